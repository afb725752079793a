// Gated feed-forward block, forward and backward, on the gfx950 matrix cores.
//
//   g = x Wg^T, u = x Wu^T, h = act(g) u, y = h Wd^T
//   dh = dy Wd, du = dh act(g), dg = dh u act'(g),
//   dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x, dWd = dy^T h
//
// One product kernel serves every line: out(m, n) = sum_k A(m, k) B(n, k), fp32
// accumulators, with either operand stored K-contiguous (rows of k) or K-strided (rows of
// m or n), so that no operand is ever transposed in memory:
//   gate    A = x,         B = Wg and Wu     both K-contiguous; 32 columns of g and the same
//                                             32 of u alternate, so one wave holds both and
//                                             its epilogue writes h (and g, u for training)
//   down    A = h,         B = Wd            both K-contiguous
//   dgate   A = dy,        B = Wd            B K-strided; epilogue reads g and u, writes dg,
//                                             du and h
//   dx      A = [dg du],   B = [Wg; Wu]      B K-strided, two segments of K
//   dW      A = [dg du] or dy, B = x or h    both K-strided
//
// Operands travel global -> LDS by the direct loads (16 bytes per lane) through a ring of
// NS stages. A K-contiguous operand lies in LDS as rows of CH chunks and its fragments are
// 16-byte reads; a K-strided one as BK rows of m (or n), and its 16-bit fragments come
// through the LDS transpose reads (ds_read_b64_tr_b16: 16 lanes read four rows of 16
// values, lane i receives column i), fp32 ones through 4-byte reads. Reads past an
// operand's last row return zero (buffer bounds); a K tail of a K-contiguous operand is
// cleared in LDS before the last slice is used.
#include <type_traits>

#include "internal.hpp"
#include "mfma_util.hpp"

namespace muon {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;

// Round to nearest even; NaN stays NaN (the hardware conversion).
__device__ __forceinline__ unsigned short to_bf16(float f) {
  return __builtin_bit_cast(unsigned short, static_cast<__bf16>(f));
}
__device__ __forceinline__ float from_bf16(unsigned short h) {
  return __uint_as_float(static_cast<unsigned int>(h) << 16);
}

// act(g) and its derivative. silu: g s(g); gelu (tanh form): g/2 (1 + tanh v),
// v = sqrt(2/pi)(g + 0.044715 g^3), with tanh v = 1 - 2 / (exp(2v) + 1).
__device__ __forceinline__ void activation(float g, int act, float& a, float& slope) {
  if (act == kActSilu) {
    const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-g * kLog2e));
    a = g * s;
    slope = s * (1.0f + g * (1.0f - s));
  } else {
    constexpr float c = 0.79788456080286535588f, b = 0.044715f;
    const float g2 = g * g;
    const float v = c * (g + b * g * g2);
    const float th = 1.0f - 2.0f * __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(2.0f * kLog2e * v) + 1.0f);
    a = 0.5f * g * (1.0f + th);
    slope = 0.5f * (1.0f + th) + 0.5f * g * (1.0f - th * th) * c * (1.0f + 3.0f * b * g2);
  }
}

template <int KIND>
__device__ __forceinline__ void mma(f32x16& acc, const u32x4& a, const u32x4& b) {
  if constexpr (KIND == KIND_BF16) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                  acc, 0, 0, 0);
  } else {
    // each lane's 16 bytes hold 4 consecutive k; four 32x32x2 steps consume them
#pragma unroll
    for (int s = 0; s < 4; ++s)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[s]), __uint_as_float(b[s]), acc, 0, 0, 0);
  }
}

// 4 consecutive elements at p, 16-bit or 32-bit; vec: p is aligned to 4 elements.
template <int KIND>
__device__ __forceinline__ void put4(void* base, int64_t at, const float (&v)[4], int n, bool vec) {
  if constexpr (KIND == KIND_F32) {
    float* p = static_cast<float*>(base) + at;
    if (vec && n >= 4) {
      *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < n) p[e] = v[e];
    }
  } else {
    unsigned short* p = static_cast<unsigned short*>(base) + at;
    if (vec && n >= 4) {
      *reinterpret_cast<u32x2*>(p) =
          u32x2{to_bf16(v[0]) | (static_cast<unsigned int>(to_bf16(v[1])) << 16),
                to_bf16(v[2]) | (static_cast<unsigned int>(to_bf16(v[3])) << 16)};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < n) p[e] = to_bf16(v[e]);
    }
  }
}
template <int KIND>
__device__ __forceinline__ void get4(const void* base, int64_t at, float (&v)[4], int n) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (KIND == KIND_F32) v[e] = e < n ? static_cast<const float*>(base)[at + e] : 0.0f;
    else v[e] = e < n ? from_bf16(static_cast<const unsigned short*>(base)[at + e]) : 0.0f;
  }
}

// Where an operand's 16-byte chunk `c` of K-strided row `k` lies in LDS (rows of R
// elements): XOR on the 64-byte (16-bit) or 128-byte (32-bit) position, so that the four
// rows of a transpose read, or the two rows of a 4-byte read, fall on different banks.
template <int KIND, int R>
__device__ __forceinline__ int swz_strided(int k, int c) {
  constexpr int CPR = R * (KIND == KIND_F32 ? 4 : 2) / 16;
  if constexpr (KIND == KIND_F32) return c ^ (((k >> 2) & 1) << 3);
  else if constexpr (CPR >= 16) return c ^ ((k & 3) << 2);
  else return c ^ (((k >> 1) & 1) << 2);
}

// The loads of one operand's slice: per-lane byte offsets of this wave's instructions.
template <int KIND, int R, int CH, int I, bool STRIDED>
struct Loader {
  static constexpr int ES = KIND == KIND_F32 ? 4 : 2;
  static constexpr int VEC = 16 / ES;
  uint32_t off[I];
  __device__ __forceinline__ void init(int wave, int lane, int64_t ld, int rows_left) {
#pragma unroll
    for (int j = 0; j < I; ++j) {
      const int at = (wave * I + j) * 64 + lane;  // chunk position in the stage
      if constexpr (STRIDED) {
        constexpr int CPR = R / VEC;
        const int k = at / CPR;
        const int c = swz_strided<KIND, R>(k, at % CPR);
        off[j] = static_cast<uint32_t>((k * ld + c * VEC) * ES);
      } else {
        const int row = at / CH;
        const int c = (at % CH) ^ swz_bits<CH>(row);
        off[j] = static_cast<uint32_t>((min(row, rows_left - 1) * ld + c * VEC) * ES);
      }
    }
  }
};

// A buffer over `elems` elements at `base` (64-bit count, clamped to what 32-bit offsets
// reach; the host keeps a tile's rows under 2^31 bytes), rounded up to a whole 16-byte
// chunk: bases and rows are 16-byte aligned, so such a chunk shares its page with a valid one.
template <int ES>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* base, int64_t elems) {
  int64_t bytes = (elems * ES + 15) & ~int64_t{15};
  bytes = bytes < 0 ? 0 : (bytes > 0x7FFFFFF0 ? 0x7FFFFFF0 : bytes);
  return make_rsrc(base, static_cast<uint32_t>(bytes));
}

// KIND: element type of x, weights and outputs. BM x BN output tile, WM x WN waves, NS LDS
// stages of CH 16-byte chunks of K. AS / BS: A / B stored K-strided.
template <int KIND, int BM, int BN, int WM, int WN, int NS, int CH, bool AS, bool BS, int EPI>
__global__ __launch_bounds__(64 * WM * WN) void ffn_gemm(const FfnGemm p) {
  constexpr int NW = WM * WN, NT = 64 * NW;
  constexpr int ES = KIND == KIND_F32 ? 4 : 2;
  constexpr int VEC = 16 / ES;
  constexpr int BK = CH * VEC;
  constexpr int TWM = BM / WM, TWN = BN / WN;
  constexpr int FM = TWM / 32, FN = TWN / 32;
  constexpr int IA = BM * CH / (64 * NW), IB = BN * CH / (64 * NW);  // loads per wave and slice
  constexpr int STAGE = (BM + BN) * CH;
  constexpr int KL = CH / 2;                                          // MFMA k-steps per slice
  constexpr int D = NS - 1;
  constexpr bool DUAL = EPI == FFN_GATE;
  static_assert(IA * 64 * NW == BM * CH && IB * 64 * NW == BN * CH, "whole instructions");
  static_assert(!DUAL || (!AS && !BS && FN % 2 == 0), "gate: K-contiguous, column pairs");
  __shared__ u32x4 lds[NS * STAGE];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // Workgroups are dealt round-robin to the 8 XCDs: give each XCD a contiguous run of the
  // logical sequence, walked in groups of 8 tile rows, so that neighbours share panels in
  // its L2.
  int tm, tn, z;
  {
    const int i = blockIdx.x, nwg = gridDim.x;
    const int xcd = i & 7, q = nwg >> 3, r = nwg & 7;
    int t = xcd * q + min(xcd, r) + (i >> 3);
    z = t / p.tiles;
    t -= z * p.tiles;
    constexpr int GM = 8;
    const int group = GM * p.tiles_n;
    const int g = t / group;
    const int first = g * GM;
    const int gm = min(p.tiles_m - first, GM);
    const int r2 = t - g * group;
    tm = first + r2 % gm;
    tn = r2 / gm;
  }
  const int batch = z / p.splits, split = z - batch * p.splits;
  const int m0 = tm * BM;
  const int n0 = DUAL ? tn * (BN / 2) : tn * BN;

  // Slices of this workgroup: [kt0, kt0 + nk) of the product's nk0 (+ nk1) slices.
  const int kt0 = split * p.slices_per_split;
  const int nk = min(p.slices - kt0, p.slices_per_split);

  const char* A[2];
  const char* Bp[2];
  A[0] = static_cast<const char*>(p.A[p.batched ? batch : 0]);
  A[1] = static_cast<const char*>(p.A[1]);
  Bp[0] = static_cast<const char*>(p.B[0]);
  Bp[1] = static_cast<const char*>(p.B[1]);

  Loader<KIND, BM, CH, IA, AS> la;
  la.init(wave, lane, p.lda, p.M - m0);
  Loader<KIND, BN, CH, IB, BS> lb;
  if constexpr (DUAL) {
    // rows 64 t .. 64 t + 31 of the tile come from Wg, the next 32 from Wu (same columns)
#pragma unroll
    for (int j = 0; j < IB; ++j) {
      const int at = (wave * IB + j) * 64 + lane;
      const int row = at / CH;
      const int c = (at % CH) ^ swz_bits<CH>(row);
      const int f = min((row >> 6) * 32 + (row & 31), p.N - n0 - 1);
      lb.off[j] = static_cast<uint32_t>((f * ((row & 32) ? p.ldb1 : p.ldb) + c * VEC) * ES);
    }
  } else {
    lb.init(wave, lane, p.ldb, p.N - n0);
  }

  auto issue = [&](int stage, int kt) {
    kt += kt0;
    const int seg = kt >= p.slices0 ? 1 : 0;
    const int64_t k0 = static_cast<int64_t>(kt - (seg ? p.slices0 : 0)) * BK;
    u32x4* sa = lds + stage * STAGE;
    u32x4* sb = sa + BM * CH;
    const char* ab = seg ? A[1] : A[0];
    const char* bb = seg ? Bp[1] : Bp[0];
    if constexpr (AS) {
      const auto r = rsrc_of<ES>(ab + (k0 * p.lda + m0) * ES, (p.K - k0 - 1) * p.lda + p.M - m0);
#pragma unroll
      for (int j = 0; j < IA; ++j) buf_load_lds(r, sa + (wave * IA + j) * 64, la.off[j], 0);
    } else {
      const auto r = rsrc_of<ES>(ab + m0 * p.lda * ES, (min(p.M - m0, BM) - 1) * p.lda + p.KA);
#pragma unroll
      for (int j = 0; j < IA; ++j) buf_load_lds(r, sa + (wave * IA + j) * 64, la.off[j], static_cast<int>(k0 * ES));
    }
    if constexpr (BS) {
      const int64_t ld = seg ? p.ldb1 : p.ldb;
      const auto r = rsrc_of<ES>(bb + (k0 * ld + n0) * ES, (p.K - k0 - 1) * ld + p.N - n0);
#pragma unroll
      for (int j = 0; j < IB; ++j) buf_load_lds(r, sb + (wave * IB + j) * 64, lb.off[j], 0);
    } else if constexpr (DUAL) {
      const int64_t last = min(p.N - n0, BN / 2) - 1;
      const auto r0 = rsrc_of<ES>(Bp[0] + n0 * p.ldb * ES, last * p.ldb + p.K);
      const auto r1 = rsrc_of<ES>(Bp[1] + n0 * p.ldb1 * ES, last * p.ldb1 + p.K);
#pragma unroll
      for (int j = 0; j < IB; ++j) {
        const bool up = ((wave * IB + j) * 64 / CH) & 32;  // one matrix per instruction (64 / CH rows)
        if (up) buf_load_lds(r1, sb + (wave * IB + j) * 64, lb.off[j], static_cast<int>(k0 * ES));
        else buf_load_lds(r0, sb + (wave * IB + j) * 64, lb.off[j], static_cast<int>(k0 * ES));
      }
    } else {
      const auto r = rsrc_of<ES>(bb + n0 * p.ldb * ES, (min(p.N - n0, BN) - 1) * p.ldb + p.K);
#pragma unroll
      for (int j = 0; j < IB; ++j) buf_load_lds(r, sb + (wave * IB + j) * 64, lb.off[j], static_cast<int>(k0 * ES));
    }
  };

  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  const int wm0 = (wave / WN) * TWM;
  const int wn0 = (wave % WN) * TWN;

  // Fragment of 32 rows starting at r0 (tile coordinates) and k-step kk: 16 bytes per lane,
  // lane l holding row r0 + l % 32 and k = (2 kk + l / 32) VEC .. + VEC - 1.
  auto frag = [&](const u32x4* s, auto strided, auto rows_tag, int r0, int kk) -> u32x4 {
    constexpr bool STR = decltype(strided)::value;
    constexpr int R = decltype(rows_tag)::value;
    if constexpr (!STR) {
      return s[swz_ch<CH>(r0 + (lane & 31), 2 * kk + (lane >> 5))];
    } else if constexpr (KIND == KIND_F32) {
      u32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = 8 * kk + 4 * (lane >> 5) + e;
        const int col = r0 + (lane & 31);
        v[e] = reinterpret_cast<const unsigned int*>(s)[(k * (R / VEC) + swz_strided<KIND, R>(k, col >> 2)) * 4 + (col & 3)];
      }
      return v;
    } else {
      u32x2 h[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int k = 16 * kk + 8 * (lane >> 5) + 4 * t + ((lane & 15) >> 2);
        const int col = r0 + ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
        const unsigned short* q =
            reinterpret_cast<const unsigned short*>(s) + (k * (R / VEC) + swz_strided<KIND, R>(k, col >> 3)) * 8 + (col & 7);
        h[t] = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                             (__attribute__((address_space(3))) s16x4*)q));
      }
      return u32x4{h[0][0], h[0][1], h[1][0], h[1][1]};
    }
  };
  using TA = std::integral_constant<bool, AS>;
  using TB = std::integral_constant<bool, BS>;
  using RA = std::integral_constant<int, BM>;
  using RB = std::integral_constant<int, BN>;
  u32x4 fa[2][FM], fb[2][FN];
  auto load_frags = [&](int buf, const u32x4* sa, int kk) {
    const u32x4* sb = sa + BM * CH;
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[buf][i] = frag(sa, TA{}, RA{}, wm0 + i * 32, kk);
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[buf][j] = frag(sb, TB{}, RB{}, wn0 + j * 32, kk);
  };

  // Ring of NS stages as in gemm.hip: slice k computes while slices k + 1 .. k + NS - 1 are
  // in flight; past the end the last slice is loaded again into a stage that is not read.
#pragma unroll
  for (int s0 = 0; s0 < D; ++s0) issue(s0, min(s0, nk - 1));
  wait_vmcnt<(D - 1) * (IA + IB)>();
  __builtin_amdgcn_s_barrier();
  issue(D, min(D, nk - 1));
  load_frags(0, lds, 0);

  constexpr int RDS = KIND == KIND_F32 ? 4 : 2;                       // LDS reads of a strided fragment
  constexpr int NRD = FM * (AS ? RDS : 1) + FN * (BS ? RDS : 1);      // LDS reads per k-step
  constexpr int NMF = (KIND == KIND_F32 ? 4 : 1) * FM * FN;           // MFMAs per k-step
  static_assert(KL % 2 == 0, "fragment buffers alternate in pairs");
  auto slice = [&](int kt, auto next_tag) {
    constexpr bool NEXT = decltype(next_tag)::value;
    const u32x4* sa = lds + (kt % NS) * STAGE;
#pragma unroll
    for (int kl = 0; kl < KL; ++kl) {
      const int cur = kl & 1;
      if (kl + 1 < KL) {
        load_frags(cur ^ 1, sa, kl + 1);
      } else if constexpr (NEXT) {
#pragma unroll
        for (int kk = 0; kk + 1 < KL; ++kk) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, NRD, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, NMF - 1, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        wait_vmcnt_lgkm0<(D - 1) * (IA + IB)>();
        __builtin_amdgcn_s_barrier();
        load_frags(cur ^ 1, lds + ((kt + 1) % NS) * STAGE, 0);
        issue(kt % NS, min(kt + NS, nk - 1));
      }
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) mma<KIND>(acc[i][j], fb[cur][j], fa[cur][i]);
    }
    if constexpr (NEXT) {
      constexpr int NL = IA + IB;
      constexpr int NP = NL < NMF ? NL : NMF;
      __builtin_amdgcn_sched_group_barrier(0x100, NRD, 0);
#pragma unroll
      for (int q = 0; q < NP; ++q) {
        __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      }
      if constexpr (NL > NP) __builtin_amdgcn_sched_group_barrier(0x010, NL - NP, 0);
      if constexpr (NMF > NP) __builtin_amdgcn_sched_group_barrier(0x008, NMF - NP, 0);
    }
  };
  for (int kt = 0; kt + 1 < nk; ++kt) slice(kt, std::true_type{});
  if constexpr (!AS || !BS) {
    // K tail of the K-contiguous operands: what lies behind K in a row is the next row, or
    // whatever the row's padding holds. Cleared in both operands, so that a NaN there does
    // not meet a zero.
    if (p.tail > 0 && kt0 + nk == p.slices) {
      u32x4* s = lds + ((nk - 1) % NS) * STAGE;
      constexpr int R0 = AS ? BM : 0, R1 = BS ? BM : BM + BN;
      __builtin_amdgcn_sched_barrier(0);
      wait_vmcnt_lgkm0<0>();
      __builtin_amdgcn_s_barrier();
      for (int at = R0 * CH + tid; at < R1 * CH; at += NT) {
        const int row = at / CH - (at / CH >= BM ? BM : 0);
        const int valid = p.tail - ((at % CH) ^ swz_bits<CH>(row)) * VEC;  // valid elements of the chunk
        if (valid >= VEC) continue;
        u32x4 v = s[at];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          if constexpr (KIND == KIND_F32) {
            if (d >= valid) v[d] = 0;
          } else {
            if (2 * d >= valid) v[d] = 0;
            else if (2 * d + 1 >= valid) v[d] &= 0xFFFFu;
          }
        }
        s[at] = v;
      }
      __syncthreads();
      load_frags(0, s, 0);
    }
  }
  slice(nk - 1, std::false_type{});
  wait_vmcnt<0>();

  // Epilogue. Lane l of block (i, j) holds row m = 32 i + l % 32 and, for q = 0..3, the four
  // columns n = 32 j + 8 q + 4 (l / 32) .. + 3.
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int m = m0 + wm0 + i * 32 + (lane & 31);
    if (m >= p.M) continue;
    if constexpr (EPI == FFN_GATE) {
#pragma unroll
      for (int j = 0; j < FN; j += 2)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int f = n0 + (wn0 + j * 32) / 2 + q * 8 + (lane >> 5) * 4;
          if (f >= p.Np) continue;
          float g[4], u[4], h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool in = f + e < p.N;  // columns behind N are the padding: zero
            g[e] = in ? acc[i][j][q * 4 + e] : 0.0f;
            u[e] = in ? acc[i][j + 1][q * 4 + e] : 0.0f;
            float slope;
            activation(g[e], p.act, h[e], slope);
            h[e] *= u[e];
          }
          const int64_t at = static_cast<int64_t>(m) * p.Np + f;
          put4<KIND>(p.C[0], at, h, 4, true);
          if (p.gu != nullptr) {
            put4<KIND_F32>(p.gu, at, g, 4, true);
            put4<KIND_F32>(p.gu + p.gu_stride, at, u, 4, true);
          }
        }
    } else if constexpr (EPI == FFN_DGATE) {
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int f = n0 + wn0 + j * 32 + q * 8 + (lane >> 5) * 4;
          if (f >= p.Np) continue;
          const int64_t at = static_cast<int64_t>(m) * p.Np + f;
          float g[4], u[4], dg[4], du[4], h[4];
          get4<KIND_F32>(p.gu, at, g, 4);
          get4<KIND_F32>(p.gu + p.gu_stride, at, u, 4);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float dh = f + e < p.N ? acc[i][j][q * 4 + e] : 0.0f;
            float a, slope;
            activation(g[e], p.act, a, slope);
            du[e] = dh * a;
            dg[e] = dh * u[e] * slope;
            h[e] = a * u[e];
          }
          put4<KIND>(p.C[0], at, dg, 4, true);
          put4<KIND>(p.C[1], at, du, 4, true);
          put4<KIND>(p.C[2], at, h, 4, true);
        }
    } else {
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int n = n0 + wn0 + j * 32 + q * 8 + (lane >> 5) * 4;
          if (n >= p.N) continue;
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = acc[i][j][q * 4 + e];
          if (p.part != nullptr) {
            put4<KIND_F32>(p.part, (static_cast<int64_t>(z) * p.M + m) * p.Np + n, v, 4, true);
            continue;
          }
          const int64_t at = static_cast<int64_t>(m) * p.ldc + n;
          if (p.c_bf16) {
            if (p.accumulate) {
              float o[4];
              get4<KIND_BF16>(p.C[batch], at, o, p.N - n);
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] += o[e];
            }
            put4<KIND_BF16>(p.C[batch], at, v, p.N - n, p.c_vec);
          } else {
            if (p.accumulate) {
              float o[4];
              get4<KIND_F32>(p.C[batch], at, o, p.N - n);
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] += o[e];
            }
            put4<KIND_F32>(p.C[batch], at, v, p.N - n, p.c_vec);
          }
        }
    }
  }
}

// Sum of the K splits' fp32 partial products in split order, then the store: one thread per
// 4 columns. HBM/L2-bound: splits x 4 bytes read per element.
__global__ __launch_bounds__(256) void ffn_join(const FfnGemm p, int64_t quads) {
  const int per_row = (p.N + 3) / 4;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < quads; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t row = i / per_row;      // batch * M + m
    const int n = static_cast<int>(i - row * per_row) * 4;
    const int batch = static_cast<int>(row / p.M);
    const int64_t m = row - static_cast<int64_t>(batch) * p.M;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < p.splits; ++s) {
      const f32x4 w = *reinterpret_cast<const f32x4*>(
          p.part + ((static_cast<int64_t>(batch) * p.splits + s) * p.M + m) * p.Np + n);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += w[e];
    }
    const int64_t at = m * p.ldc + n;
    float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (p.c_bf16) {
      if (p.accumulate) get4<KIND_BF16>(p.C[batch], at, o, p.N - n);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += o[e];
      put4<KIND_BF16>(p.C[batch], at, v, p.N - n, p.c_vec);
    } else {
      if (p.accumulate) get4<KIND_F32>(p.C[batch], at, o, p.N - n);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += o[e];
      put4<KIND_F32>(p.C[batch], at, v, p.N - n, p.c_vec);
    }
  }
}

// Copy of a rows x cols matrix whose rows are not 16-byte aligned into one whose rows are
// (ldd elements apart, zero behind cols): the product kernel's loads need whole chunks.
template <typename T>
__global__ __launch_bounds__(256) void ffn_align(const T* src, int64_t lds, T* dst, int64_t ldd, int64_t rows, int cols) {
  constexpr int VEC = 16 / sizeof(T);
  const int64_t per_row = ldd / VEC;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < rows * per_row;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t r = i / per_row;
    const int c = static_cast<int>(i - r * per_row) * VEC;
    T v[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = c + e < cols ? src[r * lds + c + e] : T(0);
    *reinterpret_cast<u32x4*>(dst + i * VEC) = *reinterpret_cast<const u32x4*>(v);
  }
}

// out (rows x cols, ld apart) <- 0: the weight gradients of no tokens.
__global__ __launch_bounds__(256) void ffn_zero(void* out, int64_t ld, int64_t rows, int64_t cols, int bf16) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < rows * cols;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t at = i / cols * ld + i % cols;
    if (bf16) static_cast<unsigned short*>(out)[at] = 0;
    else static_cast<float*>(out)[at] = 0.0f;
  }
}

template <int KIND, int BM, int BN, int WM, int WN, int NS, int CH, bool AS, bool BS, int EPI>
hipError_t launch(const FfnGemm& p, int batches, hipStream_t st) {
  const int64_t grid = static_cast<int64_t>(p.tiles) * p.splits * batches;
  if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL((ffn_gemm<KIND, BM, BN, WM, WN, NS, CH, AS, BS, EPI>), dim3(static_cast<unsigned int>(grid)),
                     dim3(64 * WM * WN), 0, st, p);
  return hipGetLastError();
}

template <int KIND, bool AS, bool BS, int EPI>
hipError_t launch_tile(int tile, const FfnGemm& p, int batches, hipStream_t st) {
  switch (tile) {
    case FFN_TILE_64x128: return launch<KIND, 64, 128, 2, 2, 3, 8, AS, BS, EPI>(p, batches, st);
    case FFN_TILE_128: return launch<KIND, 128, 128, 2, 2, 4, 8, AS, BS, EPI>(p, batches, st);
    case FFN_TILE_256:
      if constexpr (KIND != KIND_F32) return launch<KIND, 256, 256, 2, 4, 2, 8, AS, BS, EPI>(p, batches, st);
      return hipErrorInvalidValue;
  }
  return hipErrorInvalidValue;
}

template <int KIND>
hipError_t launch_kind(FfnStage stage, int tile, const FfnGemm& p, int batches, hipStream_t st) {
  switch (stage) {
    case FFN_STAGE_GATE: return launch_tile<KIND, false, false, FFN_GATE>(tile, p, batches, st);
    case FFN_STAGE_DOWN: return launch_tile<KIND, false, false, FFN_STORE>(tile, p, batches, st);
    case FFN_STAGE_DGATE: return launch_tile<KIND, false, true, FFN_DGATE>(tile, p, batches, st);
    case FFN_STAGE_DX: return launch_tile<KIND, false, true, FFN_STORE>(tile, p, batches, st);
    case FFN_STAGE_DW: return launch_tile<KIND, true, true, FFN_STORE>(tile, p, batches, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_ffn(FfnStage stage, bool f32, int tile, const FfnGemm& p, int batches, hipStream_t st) {
  hipError_t e = f32 ? launch_kind<KIND_F32>(stage, tile, p, batches, st)
                     : launch_kind<KIND_BF16>(stage, tile, p, batches, st);
  if (e != hipSuccess || p.part == nullptr) return e;
  const int64_t quads = static_cast<int64_t>(batches) * p.M * ((p.N + 3) / 4);
  const int64_t blocks = (quads + 255) / 256;
  hipLaunchKernelGGL(ffn_join, dim3(static_cast<unsigned int>(blocks < 4096 ? blocks : 4096)), dim3(256), 0, st, p, quads);
  return hipGetLastError();
}

hipError_t launch_ffn_align(const void* src, int64_t ld, void* dst, int64_t ldd, int64_t rows, int cols, bool f32,
                            hipStream_t st) {
  const int64_t chunks = rows * ldd * (f32 ? 4 : 2) / 16;
  const int64_t blocks = (chunks + 255) / 256;
  const dim3 grid(static_cast<unsigned int>(blocks < 8192 ? blocks : 8192));
  if (f32)
    hipLaunchKernelGGL(ffn_align<float>, grid, dim3(256), 0, st, static_cast<const float*>(src), ld,
                       static_cast<float*>(dst), ldd, rows, cols);
  else
    hipLaunchKernelGGL(ffn_align<unsigned short>, grid, dim3(256), 0, st, static_cast<const unsigned short*>(src), ld,
                       static_cast<unsigned short*>(dst), ldd, rows, cols);
  return hipGetLastError();
}

hipError_t launch_ffn_zero(void* out, int64_t ld, int64_t rows, int64_t cols, bool bf16, hipStream_t st) {
  const int64_t blocks = (rows * cols + 255) / 256;
  hipLaunchKernelGGL(ffn_zero, dim3(static_cast<unsigned int>(blocks < 8192 ? blocks : 8192)), dim3(256), 0, st, out, ld,
                     rows, cols, bf16 ? 1 : 0);
  return hipGetLastError();
}

}  // namespace muon
