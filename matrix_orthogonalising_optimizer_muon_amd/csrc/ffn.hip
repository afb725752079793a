// Gated feed-forward block, forward and backward, on the gfx950 matrix cores.
//
//   g = x Wg^T, u = x Wu^T, h = act(g) u, y = h Wd^T
//   dh = dy Wd, du = dh act(g), dg = dh u act'(g),
//   dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x, dWd = dy^T h
//
// One product kernel serves every line: out(m, n) = sum_k A(m, k) B(n, k), fp32
// accumulators, with either operand stored K-contiguous (rows of k) or K-strided (rows of
// m or n), so that no operand is ever transposed in memory:
//   gate    A = x,         B = Wg and Wu     both K-contiguous; 8 rows of Wg and the same 8
//                                             of Wu alternate in a tile, so one lane holds g
//                                             and u of an element and the epilogue writes h
//                                             (and g, u for training)
//   down    A = h,         B = Wd            both K-contiguous
//   dgate   A = dy,        B = Wd            B K-strided; epilogue reads g and u, writes dg,
//                                             du and h
//   dx      A = [dg du],   B = [Wg; Wu]      B K-strided, two segments of K
//   dW      A = [dg du] or dy, B = x or h    both K-strided
//
// In bf16, h, dg and du are rounded once, as operands of the next product on the bf16 matrix
// instructions (in fp32 that product would run at a tenth of the rate); g, u and all sums stay in fp32.
// Results are off by 2.3e-3 to 2.4e-3 relative to 64 bits that way, 1.6e-3 to 1.7e-3 with fp32
// intermediates and the one rounding of the result.
//
// Operands travel global -> LDS by the direct loads (16 bytes per lane) through a ring of
// NS stages. A K-contiguous operand lies in LDS as rows of CH chunks and its fragments are
// 16-byte reads; a K-strided one as BK rows of m (or n), and its 16-bit fragments come
// through the LDS transpose reads (ds_read_b64_tr_b16: 16 lanes read four rows of 16
// values, lane i receives column i), fp32 ones through 4-byte reads. Reads past an
// operand's last row return zero (buffer bounds); a K tail of a K-contiguous operand is
// cleared in LDS before the last slice is used.
#include <type_traits>
#include <utility>

#include "ffn_reads.hpp"
#include "mfma_util.hpp"
#include "train.hpp"

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
    const float g2 = fminf(g * g, 1e30f);  // finite, so that a slope of 0 or 1 stays one; NaN comes through g
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

// 16 bytes at element alignment (one instruction at any address).
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));

// Row m of one 32 x 32 block leaves in pieces of 8 columns. A lane holds columns
// 8 q + 4 (l / 32) .. + 3 for q = 0..3 of row l % 32. fp32: 16 bytes per q. bf16: lanes l
// and l + 32 swap halves, after which the lower one holds columns 8 q .. + 7 of an even q
// and the upper one of the odd q next to it: 16 bytes each.
// n: columns from the block's first to the matrix' last (more than 32: whole block).
// add: the values are added to what is there.
template <int KIND>
__device__ __forceinline__ void store_block(void* row, const float (&v)[16], int n, int half, bool add) {
  if constexpr (KIND == KIND_F32) {
    float* p = static_cast<float*>(row) + half * 4;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int left = n - q * 8 - half * 4;
      if (left >= 4) {
        f32x4 w{v[q * 4], v[q * 4 + 1], v[q * 4 + 2], v[q * 4 + 3]};
        if (add) w += __builtin_bit_cast(f32x4, static_cast<u32x4>(*reinterpret_cast<u32x4_a4*>(p + q * 8)));
        *reinterpret_cast<u32x4_a4*>(p + q * 8) = __builtin_bit_cast(u32x4, w);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < left) p[q * 8 + e] = (add ? p[q * 8 + e] : 0.0f) + v[q * 4 + e];
      }
    }
  } else {
    unsigned short* p = static_cast<unsigned short*>(row);
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
      float t[8];  // this lane's columns of q and q + 1, with the old values where they are added
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = v[q * 4 + e];
      if (add) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = q * 8 + (e >> 2) * 8 + half * 4 + (e & 3);
          if (c < n) t[e] += from_bf16(p[c]);
        }
      }
      unsigned int a[2], b[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        a[e] = to_bf16(t[2 * e]) | (static_cast<unsigned int>(to_bf16(t[2 * e + 1])) << 16);
        b[e] = to_bf16(t[4 + 2 * e]) | (static_cast<unsigned int>(to_bf16(t[5 + 2 * e])) << 16);
      }
      const auto r0 = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
      const auto r1 = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
      const u32x4 w{static_cast<unsigned int>(r0[0]), static_cast<unsigned int>(r1[0]),
                    static_cast<unsigned int>(r0[1]), static_cast<unsigned int>(r1[1])};
      const int c = (q + half) * 8;
      if (c + 8 <= n) {
        *reinterpret_cast<u32x4_a2*>(p + c) = w;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < n) p[c + e] = static_cast<unsigned short>(w[e / 2] >> (16 * (e & 1)));
      }
    }
  }
}

// The transpose read: 16 lanes read four rows of 16 values, lane i receives column i. The
// pointer is a restrict argument so that the read carries alias information: without any,
// the compiler waits for every direct load in flight before it, which empties the ring
// (7B block, 4096 tokens: dx 1094 us that way, 908 us this way; the weight gradients 1669 and
// 1505 us). What a read has to wait for is waited for by hand, as for the plain reads.
__device__ __forceinline__ u32x2 read_transposed(const __attribute__((address_space(3))) unsigned short* __restrict__ p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p));
}

// Saved g and u: fp32, in the order the lanes hold them. For 32 rows (block mb) and 8
// columns (group f8), 64 lanes x 4 values: lane l holds row l % 32, columns 4 (l / 32) .. + 3;
// g first, then u. Both kernels then move whole kilobytes.
__device__ __forceinline__ int64_t saved_at(int64_t mb, int64_t Hp, int f8, int which, int lane) {
  return ((mb * (Hp >> 3) + f8) * 2 + which) * 256 + lane * 4;
}

// Where an operand's 16-byte chunk `c` of K-strided row `k` lies in LDS (rows of R
// elements): XOR on the 64-byte (16-bit) or 128-byte (32-bit) position, so that the four
// rows of a transpose read, or the two rows of a 4-byte read, fall on different banks.
template <int KIND, int R>
__device__ __forceinline__ int swz_strided(int k, int c) {
  constexpr int CPR = R * (KIND == KIND_F32 ? 4 : 2) / 16;
  if constexpr (R == 32) return c;  // four (16-bit) or two rows to 256 bytes: apart as they are
  else if constexpr (KIND == KIND_F32) return c ^ (((k >> 2) & 1) << 3);
  else if constexpr (CPR >= 16) return c ^ ((k & 3) << 2);
  else return c ^ (((k >> 1) & 1) << 2);
}

// f(0), f(1), ..., f(N - 1) with constants.
template <int N, typename F, int... I>
__device__ __forceinline__ void each_of(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F&& f) {
  each_of<N>(f, std::make_integer_sequence<int, N>{});
}

// The product kernel. Bound by the matrix cores (at the card's power limit) for many tokens,
// by the weights' HBM traffic for few, by the fill of the ring and the epilogue where K is
// short. 7B block, 4096 tokens, 256 x 256 tiles, medians of traces on two machines: gate that saves
// g and u 1035-1131 us (984-1075 TFLOP/s), down 489-502 us (1108-1137), dgate 703-730 us (762-791; 1.1 GB
// of g, u, dg, du, h are not overlapped), dx 921-926 us (1201-1208), the weight gradients 1535-1545 us
// (1080-1087). One token, 32 x 32 tiles: 5.2 TB/s. 256 x 256 carries the most products per
// byte of LDS and L2 traffic; the small tiles exist to keep more CUs at work on small outputs,
// their k-groups to use a CU's four SIMDs on one tile.
// KIND: element type of x, weights and outputs. BM x BN output tile, WM x WN waves per
// k-group, KS k-groups (each takes its share of every slice's k-steps; their sums are joined
// through LDS), NS LDS stages of CH 16-byte chunks of K. AS / BS: A / B stored K-strided.
template <int KIND, int BM, int BN, int WM, int WN, int KS, int NS, int CH, bool AS, bool BS, int EPI>
__global__ __launch_bounds__(64 * WM * WN * KS) void ffn_gemm(const FfnGemm p) {
  constexpr int NWC = WM * WN, NW = NWC * KS, NT = 64 * NW;
  constexpr int ES = KIND == KIND_F32 ? 4 : 2;
  constexpr int VEC = 16 / ES;
  constexpr int BK = CH * VEC;
  constexpr int TWM = BM / WM, TWN = BN / WN;
  constexpr int FM = TWM / 32, FN = TWN / 32;
  constexpr int IA = BM * CH / (64 * NW), IB = BN * CH / (64 * NW);  // loads per wave and slice
  constexpr int STAGE = (BM + BN) * CH;
  constexpr int KL = CH / 2 / KS;                                     // a wave's k-steps per slice
  constexpr int D = NS - 1;
  constexpr bool DUAL = EPI == FFN_GATE;
  static_assert(IA * 64 * NW == BM * CH && IB * 64 * NW == BN * CH, "whole instructions");
  static_assert(!DUAL || (!AS && !BS && CH == 8), "gate: K-contiguous, 8 rows an instruction");
  static_assert(KL == 1 || KL % 2 == 0, "fragment buffers alternate in pairs");
  static_assert(KS == 1 || BM * BN * 4 <= NS * STAGE * 16, "the joined sums fit in LDS");
  __shared__ u32x4 lds[NS * STAGE];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kgrp = wave / NWC, wloc = wave % NWC;

  // Workgroups are dealt round-robin to the 8 XCDs: give each XCD a contiguous run of the
  // logical sequence (split, problem, tile), tiles walked in groups of 8 tile rows, so that
  // neighbours share panels in its L2.
  const void* A = p.A;
  const void* B = p.B[0];
  void* C = p.C[0];
  int64_t lda = p.lda, ldb = p.ldb, ldc = p.ldc, part0 = 0;
  int M = p.M, N = p.N, tiles_m = p.tiles_m, tiles_n = p.tiles_n;
  int tm, tn, split;
  {
    const int i = blockIdx.x, nwg = gridDim.x;
    const int xcd = i & 7, q = nwg >> 3, r = nwg & 7;
    int t = xcd * q + min(xcd, r) + (i >> 3);
    split = t / p.tiles;
    t -= split * p.tiles;
    if constexpr (AS && BS) {
      int k = 0;
      while (k + 1 < p.problems && t >= p.problem[k].tiles_m * p.problem[k].tiles_n) {
        t -= p.problem[k].tiles_m * p.problem[k].tiles_n;
        ++k;
      }
      const FfnProblem& o = p.problem[k];
      A = o.A; B = o.B; C = o.C;
      lda = o.lda; ldb = o.ldb; ldc = o.ldc; part0 = o.part0;
      M = o.M; N = o.N; tiles_m = o.tiles_m; tiles_n = o.tiles_n;
    }
    constexpr int GM = 8;
    const int group = GM * tiles_n;
    const int g = t / group;
    const int first = g * GM;
    const int gm = min(tiles_m - first, GM);
    const int r2 = t - g * group;
    tm = first + r2 % gm;
    tn = r2 / gm;
  }
  const int m0 = tm * BM;
  const int n0 = DUAL ? tn * (BN / 2) : tn * BN;

  // Slices of this workgroup: [kt0, kt0 + nk) of the product's.
  const int kt0 = split * p.slices_per_split;
  const int nk = min(p.slices - kt0, p.slices_per_split);

  // Per-lane byte offsets of this wave's load instructions: instruction j fills chunk
  // positions (wave I + j) 64 + lane of the operand's part of a stage.
  uint32_t a_off[IA], b_off[IB];
#pragma unroll
  for (int j = 0; j < IA; ++j) {
    const int at = (wave * IA + j) * 64 + lane;
    if constexpr (AS) {
      const int k = at / (BM / VEC);
      a_off[j] = static_cast<uint32_t>((k * lda + swz_strided<KIND, BM>(k, at % (BM / VEC)) * VEC) * ES);
    } else {
      const int row = at / CH;
      a_off[j] = static_cast<uint32_t>((ffn_row(row, M - m0) * lda + ((at % CH) ^ swz_bits<CH>(row)) * VEC) * ES);
    }
  }
#pragma unroll
  for (int j = 0; j < IB; ++j) {
    const int at = (wave * IB + j) * 64 + lane;
    if constexpr (BS) {
      const int k = at / (BN / VEC);
      b_off[j] = static_cast<uint32_t>((k * ldb + swz_strided<KIND, BN>(k, at % (BN / VEC)) * VEC) * ES);
    } else {
      const int row = at / CH;
      const int c = ((at % CH) ^ swz_bits<CH>(row)) * VEC;
      if constexpr (DUAL) {
        // rows 16 t .. 16 t + 7 of the tile come from Wg, the next 8 from Wu (same columns of g and u)
        const int f = ffn_row((row >> 4) * 8 + (row & 7), N - n0);
        b_off[j] = static_cast<uint32_t>((f * ((row & 8) ? p.ldb1 : ldb) + c) * ES);
      } else {
        b_off[j] = static_cast<uint32_t>((ffn_row(row, N - n0) * ldb + c) * ES);
      }
    }
  }

  // Where the next slice starts. K-contiguous: a byte offset along the rows of one buffer;
  // K-strided: a pointer, and how many rows are left. Slices are loaded in order, and up to
  // NS - 1 past the last one: those land in stages that are not read, and past an operand's
  // end they read zeros through an empty bound (ffn_reads.hpp).
  const char* a_ptr = static_cast<const char*>(A);
  const char* b_ptr = static_cast<const char*>(B);
  int a_k = 0, b_k = 0;      // K-contiguous: byte offset
  int a_rows = 0, b_rows = 0;  // K-strided: rows left
  int seg_left = 0x7FFFFFFF;   // K-strided B in two segments: slices until the second
  if constexpr (AS) {
    a_ptr += (static_cast<int64_t>(kt0) * BK * lda + m0) * ES;
    a_rows = p.K - kt0 * BK;
  } else {
    a_ptr += m0 * lda * ES;
    a_k = kt0 * BK * ES;
  }
  if constexpr (BS) {
    const bool second = p.B[1] != nullptr && kt0 >= p.slices0;
    const int s = second ? kt0 - p.slices0 : kt0;
    b_ptr = second ? static_cast<const char*>(p.B[1]) : b_ptr;
    b_ptr += (static_cast<int64_t>(s) * BK * ldb + n0) * ES;
    b_rows = p.K - s * BK;
    if (p.B[1] != nullptr && !second) seg_left = p.slices0 - kt0;
  } else {
    b_ptr += n0 * ldb * ES;
    b_k = kt0 * BK * ES;
  }
  auto bytes_of = [&](int rows, int64_t ld, int last) { return ffn_bytes(rows, ld, last, ES); };
  const int a_bytes = AS ? 0 : bytes_of(min(M - m0, BM), lda, p.KA);
  const int b_bytes = BS ? 0 : bytes_of(min(N - n0, DUAL ? BN / 2 : BN), ldb, p.K);
  const char* b1_ptr = DUAL ? static_cast<const char*>(p.B[1]) + n0 * p.ldb1 * ES : nullptr;
  const int b1_bytes = DUAL ? bytes_of(min(N - n0, BN / 2), p.ldb1, p.K) : 0;
  const int a_end = ffn_end(a_bytes, p.KA, ES), b_end = ffn_end(b_bytes, p.K, ES);

  auto issue = [&](int stage) {
    u32x4* sa = lds + stage * STAGE + wave * IA * 64;
    u32x4* sb = lds + stage * STAGE + BM * CH + wave * IB * 64;
    {
      const FfnWindow w = AS ? FfnWindow{bytes_of(min(a_rows, BK), lda, M - m0), 0} : ffn_window(a_k, a_end, a_bytes);
      const auto r = make_rsrc(a_ptr, w.bytes);
#pragma unroll
      for (int j = 0; j < IA; ++j) buf_load_lds(r, sa + j * 64, a_off[j], w.at);
      if constexpr (AS) {
        a_ptr += static_cast<int64_t>(BK * ES) * lda;
        a_rows -= BK;
      } else {
        a_k += BK * ES;
      }
    }
    const FfnWindow w = BS ? FfnWindow{bytes_of(min(b_rows, BK), ldb, N - n0), 0} : ffn_window(b_k, b_end, b_bytes);
    const auto r = make_rsrc(b_ptr, w.bytes);
    if constexpr (DUAL) {
      const FfnWindow w1 = ffn_window(b_k, b_end, b1_bytes);
      const auto r1 = make_rsrc(b1_ptr, w1.bytes);
#pragma unroll
      for (int j = 0; j < IB; ++j) {
        if ((wave * IB + j) & 1) buf_load_lds(r1, sb + j * 64, b_off[j], w1.at);
        else buf_load_lds(r, sb + j * 64, b_off[j], w.at);
      }
    } else {
#pragma unroll
      for (int j = 0; j < IB; ++j) buf_load_lds(r, sb + j * 64, b_off[j], w.at);
    }
    if constexpr (BS) {
      b_ptr += static_cast<int64_t>(BK * ES) * ldb;
      b_rows -= BK;
      if (--seg_left == 0) {
        b_ptr = static_cast<const char*>(p.B[1]) + static_cast<int64_t>(n0) * ES;
        b_rows = p.K;
      }
    } else {
      b_k += BK * ES;
    }
  };

  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  const int wm0 = (wloc / WN) * TWM;
  const int wn0 = (wloc % WN) * TWN;

  // Fragment of 32 rows starting at r0 (tile coordinates) and k-step kk: 16 bytes per lane,
  // lane l holding row r0 + l % 32 and k = (2 kk + l / 32) VEC .. + VEC - 1.
  auto frag = [&](const u32x4* s, auto strided, auto rows_tag, int r0, int kk) -> u32x4 {
    constexpr bool STR = decltype(strided)::value;
    constexpr int R = decltype(rows_tag)::value;
    if constexpr (!STR) {
      return s[swz_ch<CH>(r0 + (lane & 31), 2 * kk + half)];
    } else if constexpr (KIND == KIND_F32) {
      u32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = 8 * kk + 4 * half + e;
        const int col = r0 + (lane & 31);
        v[e] = reinterpret_cast<const unsigned int*>(s)[(k * (R / VEC) + swz_strided<KIND, R>(k, col >> 2)) * 4 + (col & 3)];
      }
      return v;
    } else {
      u32x2 h[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int k = 16 * kk + 8 * half + 4 * t + ((lane & 15) >> 2);
        const int col = r0 + ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
        const unsigned short* q =
            reinterpret_cast<const unsigned short*>(s) + (k * (R / VEC) + swz_strided<KIND, R>(k, col >> 3)) * 8 + (col & 7);
        h[t] = read_transposed((const __attribute__((address_space(3))) unsigned short*)q);
      }
      return u32x4{h[0][0], h[0][1], h[1][0], h[1][1]};
    }
  };
  using TA = std::integral_constant<bool, AS>;
  using TB = std::integral_constant<bool, BS>;
  using RA = std::integral_constant<int, BM>;
  using RB = std::integral_constant<int, BN>;
  u32x4 fa[2][FM], fb[2][FN];
  const int kk0 = kgrp * KL;
  auto load_frags = [&](int buf, const u32x4* sa, int kk) {
    const u32x4* sb = sa + BM * CH;
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[buf][i] = frag(sa, TA{}, RA{}, wm0 + i * 32, kk);
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[buf][j] = frag(sb, TB{}, RB{}, wn0 + j * 32, kk);
  };

  // Ring of NS stages as in gemm.hip: while slice k is computed, slices k + 1 .. k + NS - 1
  // are in flight or landed.
#pragma unroll
  for (int s0 = 0; s0 < D; ++s0) issue(s0);
  wait_vmcnt<(D - 1) * (IA + IB)>();
  __builtin_amdgcn_s_barrier();
  issue(D);
  load_frags(0, lds, kk0);

  constexpr int RDS = KIND == KIND_F32 ? 4 : 2;                       // LDS reads of a strided fragment
  constexpr int NRD = FM * (AS ? RDS : 1) + FN * (BS ? RDS : 1);      // LDS reads per k-step
  constexpr int NMF = (KIND == KIND_F32 ? 4 : 1) * FM * FN;           // MFMAs per k-step
  auto slice = [&](int kt, auto next_tag) {
    constexpr bool NEXT = decltype(next_tag)::value;
    const u32x4* sa = lds + (kt % NS) * STAGE;
#pragma unroll
    for (int kl = 0; kl < KL; ++kl) {
      const int cur = kl & 1;
      if (kl + 1 < KL) {
        load_frags(cur ^ 1, sa, kk0 + kl + 1);
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
        load_frags(cur ^ 1, lds + ((kt + 1) % NS) * STAGE, kk0);
        issue(kt % NS);
      }
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) mma<KIND>(acc[i][j], fb[cur][j], fa[cur][i]);
    }
    if constexpr (KL == 1) {  // one k-step a slice: the next slice's fragments move up
#pragma unroll
      for (int i = 0; i < FM; ++i) fa[0][i] = fa[1][i];
#pragma unroll
      for (int j = 0; j < FN; ++j) fb[0][j] = fb[1][j];
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
      load_frags(0, s, kk0);
    }
  }
  slice(nk - 1, std::false_type{});
  wait_vmcnt<0>();

  if constexpr (KS > 1) {
    // The k-groups' sums, added in the order of the groups.
    float* red = reinterpret_cast<float*>(lds);
    for (int g = KS - 1; g >= 1; --g) {
      __syncthreads();
      if (kgrp == g) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) red[((i * FN + j) * 16 + e) * (64 * NWC) + wloc * 64 + lane] = acc[i][j][e];
      }
      __syncthreads();
      if (kgrp == g - 1) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] += red[((i * FN + j) * 16 + e) * (64 * NWC) + wloc * 64 + lane];
      }
    }
    if (kgrp != 0) return;
  }

  // Epilogue. Lane l of block (i, j) holds row m = 32 i + l % 32 and, for q = 0..3, the four
  // columns n = 32 j + 8 q + 4 (l / 32) .. + 3. Lanes l and l + 32 share a row, so they take
  // the same branches.
  each<FM>([&](auto i_tag) {  // unrolled whatever its size: the accumulators stay in registers
    constexpr int i = decltype(i_tag)::value;
    const int m = m0 + wm0 + i * 32 + (lane & 31);
    const int64_t mb = (m0 + wm0) / 32 + i;
    if constexpr (EPI == FFN_GATE) {
      if (mb * 32 >= M) return;
      // two blocks of 16 columns each make 32 columns of h where the wave has a pair
      constexpr int PAIR = FN % 2 == 0 ? 2 : 1;
      each<FN / PAIR>([&](auto j_tag) {
        constexpr int j = decltype(j_tag)::value * PAIR;
        const int f = n0 + (wn0 + j * 32) / 2;
        if (f >= p.Np) return;
        float h[16];
#pragma unroll
        for (int t = 0; t < 2 * PAIR; ++t) {  // groups of 8 columns
          float g[4], u[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // columns behind N, and the saved rows behind M, are padding: zero
            const bool in = f + t * 8 + half * 4 + e < N && m < M;
            g[e] = in ? acc[i][j + t / 2][(t & 1) * 8 + e] : 0.0f;
            u[e] = in ? acc[i][j + t / 2][(t & 1) * 8 + 4 + e] : 0.0f;
            float a, slope;
            activation(g[e], p.act, a, slope);
            h[t * 4 + e] = a * u[e];
          }
          if (p.gu != nullptr) {
            const int64_t at = saved_at(mb, p.Np, (f >> 3) + t, 0, lane);
            *reinterpret_cast<f32x4*>(p.gu + at) = f32x4{g[0], g[1], g[2], g[3]};
            *reinterpret_cast<f32x4*>(p.gu + at + 256) = f32x4{u[0], u[1], u[2], u[3]};
          }
        }
        if constexpr (PAIR == 1) {
#pragma unroll
          for (int e = 8; e < 16; ++e) h[e] = 0.0f;
        }
        if (m < M)
          store_block<KIND>(static_cast<char*>(C) + (static_cast<int64_t>(m) * ldc + f) * ES, h, 16 * PAIR, half, false);
      });
    } else if constexpr (EPI == FFN_DGATE) {
      if (m >= M) return;
      f32x4 g[FN][4], u[FN][4];
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int f = n0 + wn0 + j * 32;
        if (f >= p.Np) continue;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t at = saved_at(mb, p.Np, (f >> 3) + q, 0, lane);
          g[j][q] = *reinterpret_cast<const f32x4*>(p.gu + at);
          u[j][q] = *reinterpret_cast<const f32x4*>(p.gu + at + 256);
        }
      }
      each<FN>([&](auto j_tag) {
        constexpr int j = decltype(j_tag)::value;
        const int f = n0 + wn0 + j * 32;
        if (f >= p.Np) return;
        float dg[16], du[16], h[16];
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float dh = f + q * 8 + half * 4 + e < N ? acc[i][j][q * 4 + e] : 0.0f;
            float a, slope;
            activation(g[j][q][e], p.act, a, slope);
            du[q * 4 + e] = dh * a;
            dg[q * 4 + e] = dh * u[j][q][e] * slope;
            h[q * 4 + e] = a * u[j][q][e];
          }
        const int64_t at = (static_cast<int64_t>(m) * ldc + f) * ES;
        store_block<KIND>(static_cast<char*>(C) + at, dg, 32, half, false);
        store_block<KIND>(static_cast<char*>(p.C[1]) + at, du, 32, half, false);
        store_block<KIND>(static_cast<char*>(p.C[2]) + (static_cast<int64_t>(m) * p.Np + f) * ES, h, 32, half, false);
      });
    } else {
      if (m >= M) return;
      each<FN>([&](auto j_tag) {
        constexpr int j = decltype(j_tag)::value;
        const int n = n0 + wn0 + j * 32;
        if (n >= N) return;
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = acc[i][j][e];
        if (p.part != nullptr)
          store_block<KIND_F32>(p.part + split * p.part_split + part0 + static_cast<int64_t>(m) * ((N + 7) & ~7) + n, v, N - n, half, false);
        else if (p.c_bf16)
          store_block<KIND_BF16>(static_cast<unsigned short*>(C) + static_cast<int64_t>(m) * ldc + n, v, N - n, half, p.accumulate);
        else
          store_block<KIND_F32>(static_cast<float*>(C) + static_cast<int64_t>(m) * ldc + n, v, N - n, half, p.accumulate);
      });
    }
  });
}

// Sum of the K splits' fp32 partial products in split order, then the store: one thread per
// 4 columns, up to 8 partials requested at a time. Bound by the reads of the partials
// (splits x 4 bytes per element: 13 us for four of 2048 x 2048), or by their latency when there are
// few (100 x 256, 16 splits: 7.0 us one partial after the other, 4.2 us this way).
__global__ __launch_bounds__(256) void ffn_join(const FfnGemm p, int64_t pieces) {
  for (int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; at < pieces; at += static_cast<int64_t>(gridDim.x) * 256) {
    void* C = p.C[0];
    int64_t ldc = p.ldc, part0 = 0, i = at;
    int N = p.N;
    if (p.problems > 0) {
      int k = 0;
      while (k + 1 < p.problems && i >= static_cast<int64_t>(p.problem[k].M) * ((p.problem[k].N + 3) / 4)) {
        i -= static_cast<int64_t>(p.problem[k].M) * ((p.problem[k].N + 3) / 4);
        ++k;
      }
      C = p.problem[k].C;
      ldc = p.problem[k].ldc;
      part0 = p.problem[k].part0;
      N = p.problem[k].N;
    }
    const int per_row = (N + 3) / 4;
    const int64_t m = i / per_row;
    const int n = static_cast<int>(i - m * per_row) * 4;
    const float* src = p.part + part0 + m * ((N + 7) & ~7) + n;
    const int64_t step = p.part_split;
    f32x4 v{0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < p.splits; s += 8) {
      f32x4 w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = *reinterpret_cast<const f32x4*>(src + min(s + k, p.splits - 1) * step);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (s + k < p.splits) v += w[k];
    }
    const int left = N - n;
    if (p.c_bf16) {
      unsigned short* c = static_cast<unsigned short*>(C) + m * ldc + n;
      unsigned short out[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (p.accumulate && e < left) v[e] += from_bf16(c[e]);
        out[e] = to_bf16(v[e]);
      }
      if (left >= 4) {
        *reinterpret_cast<u32x2_a2*>(c) = u32x2{out[0] | (static_cast<unsigned int>(out[1]) << 16),
                                                out[2] | (static_cast<unsigned int>(out[3]) << 16)};
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < left) c[e] = out[e];
      }
    } else {
      float* c = static_cast<float*>(C) + m * ldc + n;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) c[e] = (p.accumulate ? c[e] : 0.0f) + v[e];
    }
  }
}

// Copies of matrices whose rows are not 16-byte aligned into ones whose rows are (zero behind
// the last column): the product kernel's loads need whole chunks. One launch for all of a
// call's operands; a workgroup copies 256 chunks of one. Latency-bound at the sizes it meets:
// 4.4 us for the five operands of 1537 tokens, 413 x 1111 (2.8 to 3.4 us each on their own).
template <typename T>
__global__ __launch_bounds__(256) void ffn_align(const FfnCopies c) {
  constexpr int VEC = 16 / sizeof(T);
  int o = 0;
#pragma unroll
  for (int k = 1; k < FfnCopies::kMost; ++k)
    if (k < c.n && c.block0[k] <= static_cast<int64_t>(blockIdx.x)) o = k;
  const int64_t i = (blockIdx.x - c.block0[o]) * 256 + threadIdx.x;
  const int64_t per_row = c.ldd[o] / VEC;
  const int64_t r = i / per_row;
  if (r >= c.rows[o]) return;
  const int at = static_cast<int>(i - r * per_row) * VEC;
  const T* src = static_cast<const T*>(c.src[o]) + r * c.lds[o] + at;
  const int left = c.cols[o] - at;
  u32x4 v;
  if (left >= VEC) {
    v = *reinterpret_cast<const u32x4_a2*>(src);
  } else {
    T e[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) e[k] = k < left ? src[k] : T(0);
    v = __builtin_bit_cast(u32x4, e);
  }
  reinterpret_cast<u32x4*>(c.dst[o])[i] = v;
}

// out (rows x cols, ld apart) <- 0: the weight gradients of no tokens. Bound by its stores.
__global__ __launch_bounds__(256) void ffn_zero(void* out, int64_t ld, int64_t rows, int64_t cols, int bf16) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < rows * cols;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t at = i / cols * ld + i % cols;
    if (bf16) static_cast<unsigned short*>(out)[at] = 0;
    else static_cast<float*>(out)[at] = 0.0f;
  }
}

template <int KIND, int BM, int BN, int WM, int WN, int KS, int NS, int CH, bool AS, bool BS, int EPI>
hipError_t launch(const FfnGemm& p, hipStream_t st) {
  const int64_t grid = static_cast<int64_t>(p.tiles) * p.splits;
  if (grid * (64 * WM * WN * KS) > 0xFFFFFFFF) return hipErrorInvalidValue;  // threads of a launch
  hipLaunchKernelGGL((ffn_gemm<KIND, BM, BN, WM, WN, KS, NS, CH, AS, BS, EPI>), dim3(static_cast<unsigned int>(grid)),
                     dim3(64 * WM * WN * KS), 0, st, p);
  return hipGetLastError();
}

template <int KIND, bool AS, bool BS, int EPI>
hipError_t launch_tile(int tile, const FfnGemm& p, hipStream_t st) {
  switch (tile) {
    case FFN_TILE_32: return launch<KIND, 32, 32, 1, 1, 4, 8, 8, AS, BS, EPI>(p, st);
    case FFN_TILE_64: return launch<KIND, 64, 64, 2, 2, 2, 4, 8, AS, BS, EPI>(p, st);
    case FFN_TILE_64x128: return launch<KIND, 64, 128, 2, 2, 1, 3, 8, AS, BS, EPI>(p, st);
    case FFN_TILE_128: return launch<KIND, 128, 128, 2, 2, 1, 4, 8, AS, BS, EPI>(p, st);
    case FFN_TILE_128x256:
      if constexpr (KIND != KIND_F32) return launch<KIND, 128, 256, 2, 4, 1, 3, 8, AS, BS, EPI>(p, st);
      return hipErrorInvalidValue;
    case FFN_TILE_256:
      if constexpr (KIND != KIND_F32) return launch<KIND, 256, 256, 2, 4, 1, 2, 8, AS, BS, EPI>(p, st);
      return hipErrorInvalidValue;
  }
  return hipErrorInvalidValue;
}

template <int KIND>
hipError_t launch_kind(FfnStage stage, int tile, const FfnGemm& p, hipStream_t st) {
  switch (stage) {
    case FFN_STAGE_GATE: return launch_tile<KIND, false, false, FFN_GATE>(tile, p, st);
    case FFN_STAGE_DOWN: return launch_tile<KIND, false, false, FFN_STORE>(tile, p, st);
    case FFN_STAGE_DGATE: return launch_tile<KIND, false, true, FFN_DGATE>(tile, p, st);
    case FFN_STAGE_DX: return launch_tile<KIND, false, true, FFN_STORE>(tile, p, st);
    case FFN_STAGE_DW: return launch_tile<KIND, true, true, FFN_STORE>(tile, p, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_ffn(FfnStage stage, bool f32, int tile, const FfnGemm& p, hipStream_t st) {
  hipError_t e = f32 ? launch_kind<KIND_F32>(stage, tile, p, st)
                     : launch_kind<KIND_BF16>(stage, tile, p, st);
  if (e != hipSuccess || p.part == nullptr) return e;
  int64_t pieces = p.problems > 0 ? 0 : static_cast<int64_t>(p.M) * ((p.N + 3) / 4);
  for (int k = 0; k < p.problems; ++k) pieces += static_cast<int64_t>(p.problem[k].M) * ((p.problem[k].N + 3) / 4);
  const int64_t blocks = (pieces + 255) / 256;
  hipLaunchKernelGGL(ffn_join, dim3(static_cast<unsigned int>(blocks < 4096 ? blocks : 4096)), dim3(256), 0, st, p, pieces);
  return hipGetLastError();
}

hipError_t launch_ffn_align(FfnCopies& c, bool f32, hipStream_t st) {
  if (c.n == 0) return hipSuccess;
  int64_t blocks = 0;
  for (int k = 0; k < c.n; ++k) {
    c.block0[k] = blocks;
    blocks += (c.rows[k] * c.ldd[k] * (f32 ? 4 : 2) / 16 + 255) / 256;
  }
  if (blocks * 256 > 0xFFFFFFFF) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned int>(blocks));
  if (f32) hipLaunchKernelGGL(ffn_align<float>, grid, dim3(256), 0, st, c);
  else hipLaunchKernelGGL(ffn_align<unsigned short>, grid, dim3(256), 0, st, c);
  return hipGetLastError();
}

hipError_t launch_ffn_zero(void* out, int64_t ld, int64_t rows, int64_t cols, bool bf16, hipStream_t st) {
  const int64_t blocks = (rows * cols + 255) / 256;
  hipLaunchKernelGGL(ffn_zero, dim3(static_cast<unsigned int>(blocks < 8192 ? blocks : 8192)), dim3(256), 0, st, out, ld,
                     rows, cols, bf16 ? 1 : 0);
  return hipGetLastError();
}

}  // namespace muon
