// Linear attention with a decay for each head, on the gfx950 matrix cores.
//
//   S_t = e^g S_{t-1} + k_t^T v_t,   o_t = scale q_t S_t            (S: dim x dim_v, fp32)
//
// In chunks of C = 64 tokens, with Z the state before a chunk and l a token's place in it:
//   o_l = sum_{s <= l} e^{g (l - s)} (q_l . k_s) v_s + e^{g (l + 1)} q_l Z
//   Z'  = e^{g C} Z + sum_s e^{g (C - 1 - s)} k_s^T v_s
// so that every product runs on the matrix cores: 2 C (dim + dim_v) + 4 dim dim_v operations a
// token and head. The gradients are the same walk over other operands (layer.hpp), those of k
// and v from the last token to the first.
//
// A workgroup walks the chunks of one (batch, head), or of a segment of it, for a slice of dim_v
// columns. The state stays in its accumulators; only a rounded copy goes through LDS, as the operand
// of q Z. Products on 16 x 16 tiles, transposed (rows: s, dim_v or dim; columns: tokens), so that a lane's four
// results are neighbours along the axis that the next product sums over: the scores of a token become
// the operand of the product with v without leaving the lane.
//
// Bound by HBM in bf16 with enough workgroups, by the latency of a chunk's chain with few, by the fp32
// matrix instructions in fp32. MI355X, 8 x 2048 tokens, 16 heads of 128, bf16: forward 100 us for 268 MB (2.7 TB/s;
// loads and stores alone 65 us), the three gradients 240 to 255 us: 443 MB read, 197 MB
// written (2.6 TB/s), 384 workgroups of 32 chunks on 256 CUs. A 65536-token prompt of 16 heads: 156 to 195 us for
// the segments' states, 293 to 354 us for the outputs.
// In these kernels the matrix units are busy for 30 to 38% of the cycles, vector instructions run in 44 to 53%, and
// 19 to 20% of the LDS cycles are lost to bank conflicts (none in the states' walk).
//
// Steps (forward / gradients of that case, us; the sizes' first kernel took 225 / 425): state and outputs on waves of
// their own, one barrier a chunk 135 / 254; stores after the next chunk's loads 120 / 219; direct loads two
// chunks ahead, XOR-ordered rows, no spills 82 / 165 with one weighted part; then 13 and 20 us for
// accuracy: two weighted parts, scores and the state's copy in two parts, which take the error against 64 bits from 1.4
// (1.65 in gradients) to 1.0 times that of fp32 throughout. Then the copy's second part at 128 x 128 and 256 x 64
// as well (gradients 173 -> 226), three weighted parts (-> 243), a chunk's sum apart from the state (+ 3), infinities
// and NaN kept to their tokens (+ 6; forward 98 -> 103).
#include "layer.hpp"
#include "mfma_util.hpp"

namespace muon {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int C = kMixChunk;

__device__ __forceinline__ unsigned short to_bf16(float f) {
  return __builtin_bit_cast(unsigned short, static_cast<__bf16>(f));
}
__device__ __forceinline__ float from_bf16(unsigned short h) {
  return __uint_as_float(static_cast<unsigned int>(h) << 16);
}
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ unsigned int pack(float lo, float hi) {
  return __builtin_bit_cast(unsigned int, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

// What `packed` leaves of the two, rounded.
__device__ __forceinline__ unsigned int rest(unsigned int packed, float lo, float hi) {
  return pack(lo - __uint_as_float(packed << 16), hi - __uint_as_float(packed & 0xFFFF0000u));
}

template <bool F32>
struct Type {
  static constexpr int ES = F32 ? 4 : 2, VEC = 16 / ES;
  static constexpr int KF = 4 * VEC;    // products' inner extent of one fragment (four lane groups)
};

// acc += A B^T over one fragment each: lane l holds row l % 16 and a quarter (l / 16) of the
// inner extent; results: column l % 16, rows 4 (l / 16) + r.
template <bool F32>
__device__ __forceinline__ void mma(f32x4& acc, const u32x4& a, const u32x4& b) {
  if constexpr (F32) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[r]), __uint_as_float(b[r]), acc, 0, 0, 0);
  } else {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
  }
}

// LDS arrays are rows of CHUNKS 16-byte pieces, a power of two, with the pieces of row r in the order
// given by XOR with mixed(r), so that reads find different banks. (Padded rows would do, but the direct
// loads write whole kilobytes.) BY_ROWS (b where there are outputs, and the state's copy, read mostly as rows): 16-byte reads of 16 rows, which
// the hardware serves by lanes 0-3, 12-15, 20-27 and so on, each at one of two neighbouring pieces. Else (c, b of the states' walk, read as
// columns): 16-bit transpose reads of 32 bytes of 8 neighbouring rows. fp32: 4-byte reads of 64 bytes of the
// rows r, r + 4, r + 8, r + 12. One order for both kinds left a third of the LDS cycles to conflicts.
template <bool F32, int CHUNKS, bool BY_ROWS>
__device__ __forceinline__ int mixed(int r) {
  if constexpr (F32) return CHUNKS >= 16 ? r & 15 : ((r >> 2) & 1) << 2;
  if constexpr (BY_ROWS) return CHUNKS >= 16 ? r & 15 : (r >> 1) & 7;
  constexpr int SHIFT = CHUNKS >= 16 ? 0 : CHUNKS == 8 ? 1 : 2;   // rows in 256 bytes
  constexpr int PAIRS = CHUNKS >= 16 ? 7 : CHUNKS / 2 - 1;
  return (((r >> SHIFT) & PAIRS) << 1) | ((r >> 3) & 1);
}
template <bool F32, int CHUNKS, bool BY_ROWS>
__device__ __forceinline__ int piece(int r, int c) {             // its byte offset
  return (r * CHUNKS + (c ^ mixed<F32, CHUNKS, BY_ROWS>(r))) * 16;
}

// LDS accesses go through restrict pointers: without any alias information the compiler waits
// for every direct load in flight before each of them. What has to be waited for is waited for by hand.
typedef __attribute__((address_space(3))) char lds_char;
__device__ __forceinline__ u32x2 read_transposed(const lds_char* __restrict__ p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p));
}
__device__ __forceinline__ u32x4 read16(const lds_char* __restrict__ p) {
  return *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>(p);
}
__device__ __forceinline__ unsigned int read4(const lds_char* __restrict__ p) {
  return *reinterpret_cast<const __attribute__((address_space(3))) unsigned int*>(p);
}
__device__ __forceinline__ void write16(lds_char* __restrict__ p, u32x4 v) {
  *reinterpret_cast<__attribute__((address_space(3))) u32x4*>(p) = v;
}
__device__ __forceinline__ void write8(lds_char* __restrict__ p, u32x2 v) {
  *reinterpret_cast<__attribute__((address_space(3))) u32x2*>(p) = v;
}

// Where a lane reads: its part of an address is computed once, and a tile's or step's is an XOR with a
// constant (pieces of a row) and an instruction's offset (rows by sixteens). `at` is an array's offset in LDS plus the lane's part.
//
// The fragment of columns 16 t .. + 15 (as rows) over tokens, from an array of tokens. Tokens in
// the order the scores' results have: 16-bit step s: 32 s + 16 (e / 4) + 4 (l / 16) + e % 4 for
// e = 0..7; fp32: 16 s + 4 (l / 16) + e.
template <bool F32, int CHUNKS, bool BY_ROWS>
__device__ __forceinline__ int columns_lane(int lane) {
  const int g = lane >> 4, i = lane & 15;
  if constexpr (F32) return piece<true, CHUNKS, BY_ROWS>(4 * g, i >> 2) + (i & 3) * 4;
  // 16 lanes read four rows of four 8-byte pieces; lane i receives column i of the 16
  return piece<false, CHUNKS, BY_ROWS>(4 * g + (i >> 2), (i & 3) >> 1) + (i & 1) * 8;
}
template <bool F32, int CHUNKS>
__device__ __forceinline__ u32x4 columns(const lds_char* lds, int at, int t, int s) {
  u32x4 f;
  if constexpr (F32) {
#pragma unroll
    for (int r = 0; r < 4; ++r) f[r] = read4(lds + (at ^ (t << 6 | (CHUNKS >= 16 ? r << 4 : 0))) + (16 * s + r) * CHUNKS * 16);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x2 r = read_transposed(lds + (at ^ t << 5) + (32 * s + 16 * h) * CHUNKS * 16);
      f[2 * h] = r[0];
      f[2 * h + 1] = r[1];
    }
  }
  return f;
}
// The fragment of rows 16 t .. + 15 at inner step s.
template <bool F32, int CHUNKS>
__device__ __forceinline__ int rows_lane(int lane) {
  return piece<F32, CHUNKS, true>(lane & 15, lane >> 4);
}
template <int CHUNKS>
__device__ __forceinline__ u32x4 rows(const lds_char* lds, int at, int t, int s) {
  return read16(lds + (at ^ s << 6) + 16 * t * CHUNKS * 16);
}

// 16 bytes of a row from column c on.
template <bool F32>
__device__ __forceinline__ u32x4 load_whole(const char* row, int c) {
  if constexpr (F32) return *reinterpret_cast<const u32x4_a4*>(row + c * 4);
  else return *reinterpret_cast<const u32x4_a2*>(row + c * 2);
}
// Rows at any address and of any length, without a branch a load: the 16 bytes from column c on are asked for at the
// last place where they lie inside the row, and moved down when they are there. Rows of less than
// 16 bytes element by element.
template <bool F32>
struct Piece {
  static constexpr int ES = F32 ? 4 : 2, VEC = 16 / ES;
  int c, from;
  bool in, narrow;
  __device__ __forceinline__ Piece(int column, int dim)
      : c(column), from(max(min(column, dim - VEC), 0)), in(column < dim), narrow(dim < VEC) {}
  __device__ __forceinline__ u32x4 ask(const char* row, int dim) const {
    if (!narrow) return load_whole<F32>(row, from);
    u32x4 v{0, 0, 0, 0};
#pragma unroll 1
    for (int e = 0; e < dim; ++e) {              // only column 0's piece is used
      unsigned int x;
      if constexpr (F32) x = *reinterpret_cast<const unsigned int*>(row + e * 4);
      else x = static_cast<unsigned int>(*reinterpret_cast<const unsigned short*>(row + e * 2)) << (16 * (e & 1));
#pragma unroll
      for (int w = 0; w < 4; ++w) v[w] |= w == e * ES / 4 ? x : 0u;
    }
    return v;
  }
  // there: the row is one of the walk's
  __device__ __forceinline__ u32x4 take(u32x4 v, bool there) const {
    const int down = narrow ? 0 : c - from;      // elements
    if constexpr (!F32) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __builtin_amdgcn_alignbit(e < 3 ? v[e + 1] : 0u, v[e], (down & 1) * 16);
    }
    const int words = F32 ? down : down >> 1;
#pragma unroll
    for (int step = 1; step <= 2; ++step)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = words & step ? (e + step < 4 ? v[e + step] : 0u) : v[e];
    const bool here = in && there;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = here ? v[e] : 0u;
    return v;
  }
};

// N fragments from LDS in groups of G: a group is read while the one before is used. The compiler
// alone waits for each read before the product it is for, and asks for the next one after that.
template <int N, int G, typename Read, typename Use>
__device__ __forceinline__ void stream(Read&& read, Use&& use) {
  static_assert(N % G == 0, "whole groups");
  u32x4 f[2][G];
#pragma unroll
  for (int i = 0; i < G; ++i) f[0][i] = read(i);
#pragma unroll
  for (int k = 0; k < N / G; ++k) {
    if (k + 1 < N / G) {
#pragma unroll
      for (int i = 0; i < G; ++i) f[(k + 1) & 1][i] = read((k + 1) * G + i);
    }
    __builtin_amdgcn_sched_barrier(0);
    use(k * G, f[k & 1]);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// acc[t] += of the fragments f of (tile, inner step) i0 .. i0 + G - 1, tile by tile of INNER steps; inner steps
// outermost, so that neighbours in time are of different tiles.
template <bool F32, int INNER, int T, int G, int K>
__device__ __forceinline__ void products(f32x4 (&acc)[T], int i0, const u32x4 (&f)[G], const u32x4 (&b)[K]) {
#pragma unroll
  for (int s = 0; s < INNER; ++s)
#pragma unroll
    for (int i = 0; i < G; ++i)
      if ((i0 + i) % INNER == s) mma<F32>(acc[(i0 + i) / INNER], f[i], b[s]);
}

// e^{g n}, n > 0, the same for a wave, as a sum of two: a state is multiplied with the same power chunk after chunk or
// token after token, so that one fp32 number's rounding would add up over them (by 24 chunks to as much as all other roundings
// of the state).
struct Power {
  float whole, rest;
};
__device__ __forceinline__ Power power(float g, int n) {
  const double p = exp(static_cast<double>(g) * n);
  const float whole = static_cast<float>(p), rest = whole <= 3.4e38f ? static_cast<float>(p - whole) : 0.0f;
  auto uniform = [](float f) { return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(f))); };
  return {uniform(whole), uniform(rest)};
}

// Waits for this workgroup's LDS traffic and its waves. The two kinds of waves below meet here from
// loops of their own, with the same number of turns.
__device__ __forceinline__ void meet() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
}

// How a chunk's operands and the state's copy share a workgroup's LDS.
template <bool F32, int DP, int NV, bool OUT, bool DIRECT>
struct Layout {
  static constexpr int ES = F32 ? 4 : 2;
  // 16-bit: the state's copy in two parts
  static constexpr int COPY = NV * DP * ES, ZPARTS = F32 ? 1 : 2;
  static constexpr int B = C * DP * ES, CB = C * NV * ES, Z = OUT ? COPY * ZPARTS : 0;
  static constexpr int MOST = 160 * 1024;
  // copies of the operands: the next chunk's arrive (direct loads: the next two) while one is read
  static constexpr int stages(int copies) {
    return DIRECT && OUT && 3 * (B + CB) + copies * Z <= MOST ? 3 : 2 * (B + CB) + copies * Z <= MOST ? 2 : 1;
  }
  // of the state's copy: two, or one (bf16: 128 x 128 and 256 x 64) that is written again when the outputs' waves have read it
  static constexpr int COPIES = stages(2) > 1 ? 2 : 1, STAGES = stages(COPIES);
  static constexpr bool TURNS = OUT && COPIES == 1 && STAGES > 1;   // with one stage the operands' meeting does
  static constexpr int BYTES = STAGES * (B + CB) + COPIES * Z;
  static_assert(BYTES <= MOST, "LDS of a workgroup");
};

// Four waves keep the state (each dim / 4 of its rows, or half of rows and columns), with OUT four
// more make the outputs (16 of a chunk's tokens each): a SIMD then has one of either, whose matrix
// instructions, conversions and LDS reads fill each other's gaps. They meet once a chunk, and once more where the state's
// copy has one place: the outputs' waves read it first, the state's waves meet them halfway through their own products.
// DIRECT: operands whose rows are 16-byte aligned and not more than 2^29 bytes apart in a chunk (OUTSIDE below, less a reversed
// chunk's span, has to stay behind the buffer's end) go global -> LDS
// by the direct loads, issued by the state's waves up to two chunks ahead, zeros past the last row and
// column by the buffer's bounds; else all waves bring the next chunk's through registers.
template <bool F32, int DP, int NV, bool OUT, bool DIRECT>
__global__ __launch_bounds__(OUT ? 512 : 256, (OUT || Layout<F32, DP, NV, OUT, DIRECT>::BYTES <= 81920 ? 2 : 1)) void mix_walk(const MixParams p) {
  constexpr int ES = Type<F32>::ES, VEC = Type<F32>::VEC, KF = Type<F32>::KF;
  constexpr int THREADS = OUT ? 512 : 256;
  using L = Layout<F32, DP, NV, OUT, DIRECT>;
  constexpr int CHB = DP / VEC, CHC = NV / VEC;                // 16-byte pieces of a row of b (and of the state's copy), of c
  constexpr int WD = DP == 64 ? 2 : 4, WE = 4 / WD;            // waves over the state's rows and columns
  constexpr int MT = DP / WD / 16, NT = NV / WE / 16;          // its 16 x 16 tiles a wave
  constexpr int JS = C / KF;                                   // fragments over a chunk's tokens
  constexpr int DS = DP / KF;                                  // fragments over dim
  constexpr int TILES = NV / 16;
  static_assert(MT * WD * 16 == DP && NT * WE * 16 == NV, "whole tiles");
  __shared__ __attribute__((aligned(1024))) char lds_all[L::BYTES];
  lds_char* const lds = (lds_char*)lds_all;
  auto stage_of = [&](int i) { return i * (L::B + L::CB); };                       // offsets
  auto copy_of = [&](int i) { return L::STAGES * (L::B + L::CB) + i * L::Z; };

  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // Workgroups are dealt round-robin to the 8 XCDs: each XCD takes a contiguous run, in which the
  // roles and slices of a (batch, head, segment), which read the same tokens, are neighbours.
  int at;
  {
    const int i = blockIdx.x, n = gridDim.x, xcd = i & 7, q = n >> 3, r = n & 7;
    at = xcd * q + min(xcd, r) + (i >> 3);
  }
  const int which = at % p.per;
  at /= p.per;
  const int seg = at % p.walked;
  const int bh = at / p.walked;
  const int batch = bh / p.heads, head = bh % p.heads;
  int ri = 0;
  while (ri + 1 < p.roles && which >= p.role[ri + 1].first) ++ri;
  const MixRole& o = p.role[ri];
  const int e0 = (which - o.first) * NV;
  const int dim = o.dim, dim_v = o.dim_v, cols = min(dim_v - e0, NV);
  const bool rev = o.reversed;
  const int off = rev ? 0 : 1;

  int n = p.tokens;
  if (p.lengths) n = min(max(p.lengths[batch], 0), n);
  float g2 = p.log_decay[head] * kLog2e;
  g2 = g2 < -1e30f ? -1e30f : g2;                               // a decay to 0: 0^0 stays 1
  const int begin = seg * p.segment, end = min(begin + p.segment, p.tokens);
  const int live = min(end, n);                                 // places begin .. live - 1 hold tokens
  auto token = [&](int r) -> int64_t { return rev ? n - 1 - r : r; };
  auto base = [&](const MixArray& x) {
    return static_cast<const char*>(x.p) + (batch * x.sb + (head / x.group) * x.sh) * ES;
  };
  const char* rows_b = base(o.b);
  const char* rows_c = base(o.c) + e0 * ES;
  const int64_t sb = o.b.st * ES, sc = o.c.st * ES;

  // A chunk's rows of an array as a buffer: its first token in memory, and the bytes to the end of its last row.
  struct Window {
    const char* p;
    int bytes, down;   // reversed: row i of the chunk lies at (rows - 1 - i) strides
  };
  auto window = [&](const char* rows, int64_t stride, int width, int r0) -> Window {
    const int count = min(live - r0, C);
    if (count <= 0) return {rows, 0, 0};
    const int64_t first = rev ? n - r0 - count : r0;
    return {rows + first * stride, static_cast<int>((count - 1) * stride) + width * ES, rev ? static_cast<int>((count - C) * stride) : 0};
  };
  constexpr uint32_t OUTSIDE = 0x80000000u;

  // ---- b and c of a chunk through registers ----
  constexpr int LB = DIRECT ? 1 : (C * CHB + THREADS - 1) / THREADS, LC = DIRECT ? 1 : (C * CHC + THREADS - 1) / THREADS;
  static_assert(THREADS % CHB == 0 && THREADS % CHC == 0, "a thread's pieces are of one column");
  u32x4 nb[LB], nc[LC];
  const Piece<F32> piece_b(tid % CHB * VEC, dim), piece_c(tid % CHC * VEC, cols);
  auto request = [&](int r0) {
    if constexpr (!DIRECT) {
#pragma unroll
      for (int j = 0; j < LB; ++j)
        nb[j] = piece_b.ask(rows_b + token(min(r0 + tid / CHB + j * (THREADS / CHB), live - 1)) * sb, dim);
#pragma unroll
      for (int j = 0; j < LC; ++j)
        nc[j] = piece_c.ask(rows_c + token(min(r0 + tid / CHC + j * (THREADS / CHC), live - 1)) * sc, cols);
    }
  };
  auto keep = [&](int set, int r0) {
    if constexpr (!DIRECT) {
#pragma unroll
      for (int j = 0; j < LB; ++j) {
        const int r = tid / CHB + j * (THREADS / CHB);
        if (C * CHB % THREADS == 0 || r < C) write16(lds + set + piece<F32, CHB, OUT>(r, tid % CHB), piece_b.take(nb[j], r0 + r < live));
      }
#pragma unroll
      for (int j = 0; j < LC; ++j) {
        const int r = tid / CHC + j * (THREADS / CHC);
        if (C * CHC % THREADS == 0 || r < C)
          write16(lds + set + L::B + piece<F32, CHC, false>(r, tid % CHC), piece_c.take(nc[j], r0 + r < live));
      }
    }
  };

  const bool carried = o.z_in && (p.z_in_per_segment || seg == 0);

  if (!OUT || wave >= 4) {
    // ---- the state: rows d = dbase + 16 mt + .., columns e = 16 (we NT + nt) + .. ----
    const Power whole_chunk = power(p.log_decay[head], C), last_chunk = power(p.log_decay[head], max(live - begin, 0) % C);
    const int own = wave & 3, wd = own % WD, we = own / WD;
    const int dbase = wd * (DP / WD);

    // the direct loads: instruction j of this wave fills 64 pieces of b or c
    constexpr int IB = DIRECT ? C * CHB / 256 : 1, IC = DIRECT ? C * CHC / 256 : 1;
    uint32_t b_at[IB], c_at[IC];
    if constexpr (DIRECT) {
      auto from = [&](int x, int chunks, int r, int c, int64_t stride, int width) -> uint32_t {
        return c * VEC < width ? static_cast<uint32_t>((rev ? C - 1 - r : r) * static_cast<int>(stride) + c * 16) : OUTSIDE;
      };
#pragma unroll
      for (int j = 0; j < IB; ++j) {
        const int x = (own * IB + j) * 64 + lane, r = x / CHB;
        b_at[j] = from(x, CHB, r, (x % CHB) ^ mixed<F32, CHB, OUT>(r), sb, dim);
      }
#pragma unroll
      for (int j = 0; j < IC; ++j) {
        const int x = (own * IC + j) * 64 + lane, r = x / CHC;
        c_at[j] = from(x, CHC, r, (x % CHC) ^ mixed<F32, CHC, false>(r), sc, cols);
      }
    }
    auto issue = [&](int r0, int stage) {
      if constexpr (DIRECT) {
        const Window wb = window(rows_b, sb, dim, r0), wc = window(rows_c, sc, cols, r0);
        char* to = lds_all + stage * (L::B + L::CB);
        const auto fb = make_rsrc(wb.p, wb.bytes), fc = make_rsrc(wc.p, wc.bytes);
#pragma unroll
        for (int j = 0; j < IB; ++j) buf_load_lds(fb, to + (own * IB + j) * 1024, b_at[j] + wb.down, 0);
#pragma unroll
        for (int j = 0; j < IC; ++j) buf_load_lds(fc, to + L::B + (own * IC + j) * 1024, c_at[j] + wc.down, 0);
      }
    };
    constexpr int AHEAD = L::STAGES > 1 ? L::STAGES - 1 : 1;     // with one stage: after everyone has read the last chunk
    if constexpr (DIRECT) {
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) issue(begin + k * C, k);
    } else if (begin < live) {
      request(begin);
    }

    f32x4 z[MT][NT];
    {
      const float* src = nullptr;
      if (carried) src = o.z_in + (p.z_in_per_segment ? static_cast<int64_t>(bh) * p.segments + seg : bh) * dim * dim_v;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int e = 16 * (we * NT + nt) + l16;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int d = dbase + 16 * mt + 4 * g + r;
            z[mt][nt][r] = src && d < dim && e < cols ? src[d * o.z_row + (e0 + e) * o.z_col] : 0.0f;
          }
        }
    }
    // its copy for the outputs, dim_v x dim. 16-bit: rounded to bf16, as the operand of q Z, and the rest in a second
    // part (error of o against 64 bits 1.35 times that of fp32 throughout without it)
    const int z_lane = F32 ? piece<true, CHB, true>(l16, g) : piece<false, CHB, true>(l16, g >> 1) + (g & 1) * 8;
    auto show = [&](int copy) {
      if constexpr (OUT) {
        const int at = (copy + z_lane) ^ dbase * ES;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            lds_char* const to = lds + (at ^ 16 * mt * ES) + 16 * (we * NT + nt) * CHB * 16;
            if constexpr (F32) write16(to, __builtin_bit_cast(u32x4, z[mt][nt]));
            else {
              const u32x2 w{pack(z[mt][nt][0], z[mt][nt][1]), pack(z[mt][nt][2], z[mt][nt][3])};
              write8(to, w);
              write8(to + L::COPY, u32x2{rest(w[0], z[mt][nt][0], z[mt][nt][1]), rest(w[1], z[mt][nt][2], z[mt][nt][3])});
            }
          }
      }
    };
    const int b_lane = columns_lane<F32, CHB, OUT>(lane) ^ dbase * ES, c_lane = columns_lane<F32, CHC, false>(lane) ^ we * NT * 16 * ES;
    // the weights of a chunk's tokens, in the order of `columns`
    float weight[JS][VEC];
    auto weigh = [&](int rows) {
#pragma unroll
      for (int s = 0; s < JS; ++s)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int j = F32 ? 16 * s + 4 * g + e : 32 * s + 16 * (e >> 2) + 4 * g + (e & 3);
          weight[s][e] = __builtin_amdgcn_exp2f(g2 * max(rows - off - j, 0)) * o.u_scale;
        }
    };
    weigh(C);
    Power over = whole_chunk;

    if (begin < live) {
      keep(stage_of(0), begin);
      show(copy_of(0));
    }
    int stage = 0, copy = 0;
    for (int r0 = begin; r0 < live; r0 += C) {
      if constexpr (DIRECT) wait_vmcnt<(AHEAD - 1) * (IB + IC)>();   // this chunk's are in, the next one's may be on their way
      meet();
      const int set_b = stage_of(stage) + b_lane, set_c = stage_of(stage) + L::B + c_lane;
      const bool more = r0 + C < live;
      if constexpr (DIRECT && L::STAGES > 1) issue(r0 + AHEAD * C, stage + AHEAD < L::STAGES ? stage + AHEAD : stage + AHEAD - L::STAGES);
      else if (!DIRECT && more) request(r0 + C);
      const int rows = min(live - r0, C);
      if (rows < C) {
        weigh(rows);
        over = last_chunk;
      }
      // Weighted b of this wave's rows, 32 rows at a time. 16-bit: in three parts, each the rest of
      // the ones before rounded as the product's operand: their sum has the weighted value's 24 bits, so that the state is
      // one of fp32 terms (two parts, where no state leaves: 230 instead of 242 us for the gradients of 8 x 2048 tokens)
      // A tile's sum over the chunk stands apart and is added once: products summed onto the state itself each round at
      // its size (error of fp32 states against 64 bits over 24 chunks 6.9e-7 instead of 1.7e-7, with the power's rest)
      {
        // Rows of a state of 16 tiles a wave 16 at a time where the next chunk's operands wait in registers too: 32 would
        // spill (32768 tokens, 16 heads of 251 x 250: 1550 instead of 1190 us)
        constexpr int PARTS = F32 ? 1 : 3, PAIR = !DIRECT && MT * NT >= 16 ? 1 : 2;
        constexpr int N = NT * JS, G = N < 4 ? N : 4, GROUPS = MT / PAIR * (N / G);   // fragments of c, in groups of whole tiles
        static_assert(G % JS == 0, "whole tiles");
#pragma unroll
        for (int m0 = 0; m0 < MT; m0 += PAIR) {
          u32x4 kf[JS][PARTS][PAIR];
#pragma unroll
          for (int s = 0; s < JS; ++s)
#pragma unroll
            for (int mt = 0; mt < PAIR; ++mt) {
              const u32x4 f = columns<F32, CHB>(lds, set_b, m0 + mt, s);
              if constexpr (F32) {
#pragma unroll
                for (int e = 0; e < 4; ++e) kf[s][0][mt][e] = __float_as_uint(__uint_as_float(f[e]) * weight[s][e]);
              } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  float lo = __uint_as_float(f[e] << 16) * weight[s][2 * e];
                  float hi = __uint_as_float(f[e] & 0xFFFF0000u) * weight[s][2 * e + 1];
#pragma unroll
                  for (int q = 0; q < PARTS; ++q) {
                    const unsigned int w = pack(lo, hi);
                    kf[s][q][mt][e] = w;
                    lo -= __uint_as_float(w << 16);
                    hi -= __uint_as_float(w & 0xFFFF0000u);
                  }
                }
              }
            }
          stream<N, G>([&](int i) { return columns<F32, CHC>(lds, set_c, i / JS, i % JS); },
                       [&](int i0, const u32x4 (&v)[G]) {
                         if constexpr (L::TURNS) {
                           if (more && m0 / PAIR * (N / G) + i0 / G == GROUPS / 2) meet();
                         }
                         f32x4 u[PAIR][G / JS];
#pragma unroll
                         for (int mt = 0; mt < PAIR; ++mt)
#pragma unroll
                           for (int i = 0; i < G / JS; ++i) u[mt][i] = z[m0 + mt][i0 / JS + i] * over.rest;
#pragma unroll
                         for (int s = 0; s < JS; ++s)
#pragma unroll
                           for (int q = 0; q < PARTS; ++q)
#pragma unroll
                             for (int i = 0; i < G / JS; ++i)
#pragma unroll
                               for (int mt = 0; mt < PAIR; ++mt) mma<F32>(u[mt][i], kf[s][q][mt], v[i * JS + s]);
#pragma unroll
                         for (int mt = 0; mt < PAIR; ++mt)
#pragma unroll
                           for (int i = 0; i < G / JS; ++i) z[m0 + mt][i0 / JS + i] = z[m0 + mt][i0 / JS + i] * over.whole + u[mt][i];
                       });
        }
      }
      stage = stage + 1 < L::STAGES ? stage + 1 : 0;
      copy = L::COPIES - 1 - copy;
      if (more) {
        if constexpr (L::STAGES == 1) {
          meet();
          issue(r0 + C, 0);
        }
        keep(stage_of(stage), r0 + C);
        show(copy_of(copy));
      }
    }
    if constexpr (DIRECT) wait_vmcnt<0>();   // none into the LDS of a workgroup that has ended

    if (o.z_out && (p.z_out_per_segment || seg == (n > 0 ? (n - 1) / p.segment : 0))) {
      float* dst = o.z_out + (p.z_out_per_segment ? static_cast<int64_t>(bh) * p.segments + seg : bh) * dim * dim_v;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int e = 16 * (we * NT + nt) + l16;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int d = dbase + 16 * mt + 4 * g + r;
            if (d < dim && e < cols) dst[static_cast<int64_t>(d) * dim_v + e0 + e] = z[mt][nt][r];
          }
        }
    }
  }

  if (OUT && wave < 4) {
    // ---- the outputs of tokens 16 wave .. + 15 of each chunk; a lane's token is a column of the products ----
    const int i_tok = 16 * wave + l16;
    const char* rows_a = base(o.a);
    const int64_t sa = o.a.st * ES;
    constexpr bool AHEAD = DS <= 8;                             // registers for the next chunk's too
    // Fragments in a group; four where eight would spill (4 x 2309 tokens, 16 heads of 227 x 224: 253 instead of 308 us)
    constexpr int GN = DS <= (DIRECT ? 8 : 4) ? 8 : 4;
    u32x4 na[DS];
    uint32_t a_at = 0;
    if constexpr (DIRECT) a_at = static_cast<uint32_t>((rev ? C - 1 - i_tok : i_tok) * static_cast<int>(sa)) + g * 16;
    auto request_a = [&](int r0) {
      if constexpr (DIRECT) {
        const Window w = window(rows_a, sa, dim, r0);
        const auto f = make_rsrc(w.p, w.bytes);
#pragma unroll
        for (int s = 0; s < DS; ++s)
          na[s] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(f, KF * s + VEC * g < dim ? a_at + w.down + KF * s * ES : OUTSIDE, 0, 0));
      } else {
        const char* row = rows_a + token(min(r0 + i_tok, live - 1)) * sa;
#pragma unroll
        for (int s = 0; s < DS; ++s) na[s] = Piece<F32>(KF * s + VEC * g, dim).ask(row, dim);
      }
    };
    // e^{g (i - s)} of the scores' tiles, 0 above the diagonal. All four tiles are computed by every wave: without
    // branches their LDS reads and products overlap
    float within[4][4];
#pragma unroll
    for (int jt = 0; jt < 4; ++jt)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = i_tok - (16 * jt + 4 * g + r);
        within[jt][r] = d < 0 ? 0.0f : __builtin_amdgcn_exp2f(g2 * d) * o.p_scale;
      }
    const float reach = __builtin_amdgcn_exp2f(g2 * (i_tok + off)) * o.o_scale;
    const int64_t o_row = static_cast<int64_t>(p.heads) * dim_v;   // elements from token to token of the output
    const int64_t o_at = (static_cast<int64_t>(batch) * p.tokens * p.heads + head) * dim_v + e0;

    if (begin < live) {
      if constexpr (AHEAD) request_a(begin);
      request(begin);
      keep(stage_of(0), begin);
    }
    constexpr int PARTS = F32 ? 1 : 2;                          // of the scores
    auto causal = [&](f32x4 (&y)[TILES], const u32x4 (&score)[PARTS][JS], int set_c, int here) {
      asm volatile("" : "+v"(set_c));                           // addresses of its own: those of the products would stay in registers
      u32x4 ones[JS];                                           // a token's own and those before it, as `columns` orders them
#pragma unroll
      for (int s = 0; s < JS; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (F32) ones[s][e] = here < 16 * s + 4 * g + e ? 0u : 0x3F800000u;
          else {
            const int j = 32 * s + 16 * (e >> 1) + 4 * g + 2 * (e & 1);
            ones[s][e] = (here < j ? 0u : 0x3F80u) | (here < j + 1 ? 0u : 0x3F800000u);
          }
        }
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        f32x4 sum{0, 0, 0, 0}, count{0, 0, 0, 0};
        u32x4 v[JS];
#pragma unroll
        for (int s = 0; s < JS; ++s) {
          v[s] = columns<F32, CHC>(lds, set_c, t, s);
          u32x4 odd;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (F32) {
              const bool finite = (v[s][e] & 0x7F800000u) != 0x7F800000u;
              odd[e] = finite ? 0u : 0x3F800000u;
              v[s][e] = finite ? v[s][e] : 0u;
            } else {
              const bool lo = (v[s][e] & 0x7F80u) != 0x7F80u, hi = (v[s][e] & 0x7F800000u) != 0x7F800000u;
              odd[e] = (lo ? 0u : 0x3F80u) | (hi ? 0u : 0x3F800000u);
              v[s][e] &= (lo ? 0xFFFFu : 0u) | (hi ? 0xFFFF0000u : 0u);
            }
          }
          mma<F32>(count, odd, ones[s]);
        }
#pragma unroll
        for (int q = 0; q < PARTS; ++q)                           // in the order of the sums without it
#pragma unroll
          for (int s = 0; s < JS; ++s) mma<F32>(sum, v[s], score[q][s]);
#pragma unroll
        for (int r = 0; r < 4; ++r) y[t][r] = count[r] > 0.0f ? __builtin_nanf("") : sum[r];
      }
    };
    const int n_lane = rows_lane<F32, CHB>(lane), c_lane = columns_lane<F32, CHC, false>(lane);
    int stage = 0, copy = 0;
    for (int r0 = begin; r0 < live; r0 += C) {
      meet();
      const int set_n = stage_of(stage) + n_lane, set_c = stage_of(stage) + L::B + c_lane;
      const bool more = r0 + C < live;
      if constexpr (!AHEAD) request_a(r0);
      u32x4 a[DS];
#pragma unroll
      for (int s = 0; s < DS; ++s) a[s] = DIRECT ? na[s] : Piece<F32>(KF * s + VEC * g, dim).take(na[s], r0 + i_tok < live);
      if constexpr (AHEAD && DIRECT) request_a(r0 + C);          // past the last chunk: zeros
      if (more) {
        request(r0 + C);
        if constexpr (AHEAD && !DIRECT) request_a(r0 + C);
      }
      f32x4 x[TILES];
#pragma unroll
      for (int t = 0; t < TILES; ++t) x[t] = f32x4{0, 0, 0, 0};
      if (carried || r0 > begin) {
        const int z = copy_of(copy) + n_lane;
        constexpr int GZ = TILES * DS < GN ? TILES * DS : GN;
        stream<TILES * DS, GZ>([&](int i) { return rows<CHB>(lds, z, i / DS, i % DS); },
                               [&](int i0, const u32x4 (&k)[GZ]) { products<F32, DS>(x, i0, k, a); });
        if constexpr (!F32)
          stream<TILES * DS, GZ>([&](int i) { return rows<CHB>(lds, z + L::COPY, i / DS, i % DS); },
                                 [&](int i0, const u32x4 (&k)[GZ]) { products<F32, DS>(x, i0, k, a); });
      }
      if constexpr (L::TURNS) {
        if (more) meet();
      }
      // scores, transposed: rows s, columns this wave's tokens
      // 16-bit: rounded as the operand of the product with v, in two parts
      u32x4 score[PARTS][JS];
      int here = i_tok;
      {
        f32x4 sc4[4];
        asm volatile("" : "+v"(here));                             // compared here: 16 masks kept over the loop would spill
#pragma unroll
        for (int jt = 0; jt < 4; ++jt) sc4[jt] = f32x4{0, 0, 0, 0};
        stream<4 * DS, GN>([&](int i) { return rows<CHB>(lds, set_n, i / DS, i % DS); },
                          [&](int i0, const u32x4 (&k)[GN]) { products<F32, DS>(sc4, i0, k, a); });
#pragma unroll
        for (int jt = 0; jt < 4; ++jt)
#pragma unroll
          for (int r = 0; r < 4; ++r) sc4[jt][r] = here < 16 * jt + 4 * g + r ? 0.0f : sc4[jt][r] * within[jt][r];
#pragma unroll
        for (int s = 0; s < JS; ++s) {
          if constexpr (F32) {
            score[0][s] = __builtin_bit_cast(u32x4, sc4[s]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float lo = sc4[2 * s + e / 2][e % 2 * 2], hi = sc4[2 * s + e / 2][e % 2 * 2 + 1];
              score[0][s][e] = pack(lo, hi);
              score[PARTS - 1][s][e] = rest(score[0][s][e], lo, hi);
            }
          }
        }
      }
      f32x4 y[TILES];                                            // apart, as the state's sums are
#pragma unroll
      for (int t = 0; t < TILES; ++t) y[t] = f32x4{0, 0, 0, 0};
      constexpr int G = TILES * JS < GN ? TILES * JS : GN;
      stream<TILES * JS, G>([&](int i) { return columns<F32, CHC>(lds, set_c, i / JS, i % JS); },
                            [&](int i0, const u32x4 (&v)[G]) {
#pragma unroll
                              for (int q = 0; q < PARTS; ++q) products<F32, JS>(y, i0, v, score[q]);
                            });
      // A row of c that is not finite belongs to its token and those after it, but 0 times it is NaN in the sums of the
      // tokens before. Where a sum is not finite, all are made again without such elements, which are counted up to each
      // token by products of ones instead.
      float odd = 0.0f;
#pragma unroll
      for (int t = 0; t < TILES; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) odd = __builtin_fmaf(y[t][r], 0.0f, odd);
      if (__any(!(odd == 0.0f))) causal(y, score, set_c, here);
#pragma unroll
      for (int t = 0; t < TILES; ++t) x[t] = x[t] * reach + y[t];
      stage = stage + 1 < L::STAGES ? stage + 1 : 0;
      copy = L::COPIES - 1 - copy;
      if (more) {
        if constexpr (L::STAGES == 1) meet();
        keep(stage_of(stage), r0 + C);
      }
      // After the next chunk's loads are in: waiting for those does not wait for these stores. A lane holds
      // columns 16 t + 4 g .. + 3 of its token.
      const int64_t o_tok = o_at + token(r0 + i_tok) * o_row;
      if (r0 + i_tok < live) {
        if (F32 || o.out_f32) {
#pragma unroll
          for (int t = 0; t < TILES; ++t) {
            float* out = static_cast<float*>(o.out) + o_tok + 16 * t + 4 * g;
            const int left = cols - (16 * t + 4 * g);
            if (left >= 4) *reinterpret_cast<u32x4_a4*>(out) = __builtin_bit_cast(u32x4, x[t]);
            else
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (r < left) out[r] = x[t][r];
          }
        } else {
#pragma unroll
          for (int t = 0; t < TILES; t += 2) {
            // lane groups 1 and 3 of the even tile change places with 0 and 2 of the odd one: eight columns each
            const auto lo = __builtin_amdgcn_permlane16_swap(pack(x[t][0], x[t][1]), pack(x[t + 1][0], x[t + 1][1]), false, false);
            const auto hi = __builtin_amdgcn_permlane16_swap(pack(x[t][2], x[t][3]), pack(x[t + 1][2], x[t + 1][3]), false, false);
            const int c = 16 * (t + (g & 1)) + 8 * (g >> 1), left = cols - c;
            unsigned short* out = static_cast<unsigned short*>(o.out) + o_tok + c;
            const u32x4 w{static_cast<unsigned int>(lo[0]), static_cast<unsigned int>(hi[0]), static_cast<unsigned int>(lo[1]),
                          static_cast<unsigned int>(hi[1])};
            if (left >= 8) *reinterpret_cast<u32x4_a2*>(out) = w;
            else
#pragma unroll
              for (int r = 0; r < 8; ++r)
                if (r < left) out[r] = static_cast<unsigned short>(w[r / 2] >> (16 * (r & 1)));
          }
        }
      }
    }
    // rows behind the last token: zeros
    const int first = max(live, begin);
    const int64_t count = static_cast<int64_t>(end - first) * cols;
    for (int64_t x = tid; x < count; x += 256) {
      const int64_t w = o_at + (first + x / cols) * o_row + x % cols;
      if (F32 || o.out_f32) static_cast<float*>(o.out)[w] = 0.0f;
      else static_cast<unsigned short*>(o.out)[w] = 0;
    }
  }
}

// Sums of segments to the state before each: Z_{s+1} = e^{g len_s} Z_s + sum_s. One thread an
// element, segments in order; the next sums are requested ahead.
__global__ __launch_bounds__(256) void mix_scan(const MixScan p) {
  const auto o = p.one[blockIdx.z];
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= o.n) return;
  for (int bh = blockIdx.y; bh < p.batch * p.heads; bh += gridDim.y) {
    int n = p.tokens;
    if (p.lengths) n = min(max(p.lengths[bh / p.heads], 0), n);
    const float g = p.log_decay[bh % p.heads];
    const Power full = power(g, p.segment);
    float* z = o.z + static_cast<int64_t>(bh) * p.segments * o.n + i;
    float s = o.z0 ? o.z0[static_cast<int64_t>(bh) * o.n + i] : 0.0f;
    constexpr int U = 8;
    for (int k0 = 0; k0 < p.segments; k0 += U) {
      float u[U];
#pragma unroll
      for (int k = 0; k < U; ++k) u[k] = k0 + k + 1 < p.segments ? z[static_cast<int64_t>(k0 + k) * o.n] : 0.0f;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (k0 + k >= p.segments) break;
        const int len = min(max(n - (k0 + k) * p.segment, 0), p.segment);
        z[static_cast<int64_t>(k0 + k) * o.n] = s;
        if (len > 0) {                                           // behind the last token u is 0
          const Power over = len == p.segment ? full : power(g, len);
          s = over.whole * s + (over.rest * s + u[k]);
        }
      }
    }
  }
}

// Gradients of shared heads: the group's fp32 partial sums in head order, rounded once. A thread takes four
// columns and asks for four heads at once. 8 x 2048 tokens, 16 heads of 128 over 4: 56 us for dk and dv (one column a
// thread, 64-bit divisions 88 us).
__global__ __launch_bounds__(256) void mix_share(const MixShare p) {
  const auto o = p.one[blockIdx.y];
  int shift = 0;                                               // 2^shift threads across a row
  while ((4 << shift) < o.dim) ++shift;
  const int d = (threadIdx.x & ((1 << shift) - 1)) * 4, live = o.dim - d;
  if (live <= 0) return;
  const int64_t n = p.rows * p.kv_heads, each = 256 >> shift;
  for (int64_t row = blockIdx.x * each + (threadIdx.x >> shift); row < n; row += gridDim.x * each) {
    const float* q = o.part + row * p.group * o.dim + d;
    auto load = [&](int k) -> f32x4 {
      const float* x = q + static_cast<int64_t>(k) * o.dim;
      if (live >= 4) return __builtin_bit_cast(f32x4, static_cast<u32x4>(*reinterpret_cast<const u32x4_a4*>(x)));
      return f32x4{x[0], live > 1 ? x[1] : 0.0f, live > 2 ? x[2] : 0.0f, 0.0f};
    };
    f32x4 s = load(0);
    for (int k = 1; k < p.group; k += 4) {
      f32x4 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = load(min(k + j, p.group - 1));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (k + j < p.group) s += x[j];
      }
    }
    if (p.bf16) {
      unsigned short* out = static_cast<unsigned short*>(o.out) + row * o.dim + d;
      if (live >= 4) {
        *reinterpret_cast<u32x2_a2*>(out) = u32x2{pack(s[0], s[1]), pack(s[2], s[3])};
      } else {
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          if (j < live) out[j] = to_bf16(s[j]);
        }
      }
    } else {
      float* out = static_cast<float*>(o.out) + row * o.dim + d;
      if (live >= 4) {
        *reinterpret_cast<u32x4_a4*>(out) = __builtin_bit_cast(u32x4, s);
      } else {
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          if (j < live) out[j] = s[j];
        }
      }
    }
  }
}

// One token: S' = e^g S + k^T v, o = scale q S'. Bound by the state's traffic, read and written
// once: 128 requests of 28 heads of 128 x 128 90 us, 5.2 TB/s; 16 heads 5.0 us; 64 requests of 32 heads of 250 x 250 219 us,
// 4.7 TB/s (64 columns a workgroup: 437 us). A workgroup takes `lanes` threads of four
// columns across and as many rows as there are threads at a time, four of them in flight; their sums are joined in LDS in
// row order. A thread behind the last whole four columns reads the last four of the row and keeps its own.
template <bool F32>
__device__ __forceinline__ float load_one(const void* p, int64_t i) {
  if constexpr (F32) return static_cast<const float*>(p)[i];
  else return from_bf16(static_cast<const unsigned short*>(p)[i]);
}
template <bool F32>
__global__ __launch_bounds__(256) void mix_step(const MixStep p) {
  __shared__ float qk[2][256];
  __shared__ f32x4 sums[256];
  const int tid = threadIdx.x, bh = blockIdx.x, b = bh / p.heads, h = bh % p.heads;
  if (tid < p.dim) {
    qk[0][tid] = load_one<F32>(p.q, b * p.q_sb + h * p.q_sh + tid) * p.scale;
    qk[1][tid] = load_one<F32>(p.k, b * p.k_sb + (h / p.group) * p.k_sh + tid);
  }
  const int across = tid % p.lanes, down = tid / p.lanes, rows = 256 / p.lanes;
  const int e = (blockIdx.y * p.lanes + across) * 4;
  const Power decay = power(p.log_decay[h], 1);                 // token after token the same
  const int left = down < rows ? p.dim_v - e : 0;
  const int skip = left >= 4 ? 0 : 4 - left;                    // of the four columns from e - skip on: a neighbour's
  const bool four = left > 0 && p.dim_v >= 4;
  f32x4 v{0, 0, 0, 0}, acc{0, 0, 0, 0};
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (left > 0 && (four || r >= skip)) v[r] = load_one<F32>(p.v, b * p.v_sb + (h / p.group) * p.v_sh + e - skip + r);
  __syncthreads();
  const int64_t at = static_cast<int64_t>(bh) * p.dim * p.dim_v + e - skip;
  if (left > 0) {
    constexpr int U = 4;
    for (int d0 = down; d0 < p.dim; d0 += U * rows) {
      f32x4 s[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int d = min(d0 + u * rows, p.dim - 1);
        const float* z = p.z_in + at + static_cast<int64_t>(d) * p.dim_v;
        if (four) {
          s[u] = __builtin_bit_cast(f32x4, static_cast<u32x4>(*reinterpret_cast<const u32x4_a4*>(z)));
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) s[u][r] = r >= skip ? z[r] : 0.0f;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int d = d0 + u * rows;
        if (d >= p.dim) break;
        s[u] = s[u] * decay.whole + (s[u] * decay.rest + v * qk[1][d]);
        acc += s[u] * qk[0][d];
        float* z = p.z_out + at + static_cast<int64_t>(d) * p.dim_v;
        if (skip == 0) {
          *reinterpret_cast<u32x4_a4*>(z) = __builtin_bit_cast(u32x4, s[u]);
        } else {
#pragma unroll
          for (int r = 1; r < 4; ++r)
            if (r >= skip) z[r] = s[u][r];
        }
      }
    }
  }
  sums[tid] = acc;
  __syncthreads();
  if (down == 0 && left > 0) {
    for (int k = 1; k < rows; ++k) acc += sums[k * p.lanes + across];
    const int64_t x = static_cast<int64_t>(bh) * p.dim_v + e - skip;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (r >= skip) {
        if constexpr (F32) static_cast<float*>(p.out)[x + r] = acc[r];
        else static_cast<unsigned short*>(p.out)[x + r] = to_bf16(acc[r]);
      }
  }
}

template <bool F32, int DP, int NV, bool DIRECT>
hipError_t walk(bool out, const MixParams& p, int64_t groups, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(groups));
  if (out) mix_walk<F32, DP, NV, true, DIRECT><<<grid, 512, 0, st>>>(p);
  else mix_walk<F32, DP, NV, false, DIRECT><<<grid, 256, 0, st>>>(p);
  return hipGetLastError();
}
template <bool F32, int DP, int NV>
hipError_t walk(bool out, const MixParams& p, int64_t groups, hipStream_t st) {
  return p.direct ? walk<F32, DP, NV, true>(out, p, groups, st) : walk<F32, DP, NV, false>(out, p, groups, st);
}
template <bool F32>
hipError_t walk(MixTile t, bool out, const MixParams& p, int64_t groups, hipStream_t st) {
  if (t.dim == 64) return t.dim_v == 64 ? walk<F32, 64, 64>(out, p, groups, st) : walk<F32, 64, 32>(out, p, groups, st);
  if (t.dim == 128) {
    if constexpr (!F32)
      if (t.dim_v == 128) return walk<F32, 128, 128>(out, p, groups, st);
    return t.dim_v == 64 ? walk<F32, 128, 64>(out, p, groups, st) : walk<F32, 128, 32>(out, p, groups, st);
  }
  return t.dim_v == 64 ? walk<F32, 256, 64>(out, p, groups, st) : walk<F32, 256, 32>(out, p, groups, st);
}

}  // namespace

hipError_t launch_mix(bool f32, MixTile t, bool out, const MixParams& p, int64_t groups, hipStream_t st) {
  return f32 ? walk<true>(t, out, p, groups, st) : walk<false>(t, out, p, groups, st);
}

hipError_t launch_mix_scan(const MixScan& p, hipStream_t st) {
  int most = 0;
  for (int i = 0; i < p.count; ++i) most = p.one[i].n > most ? p.one[i].n : most;
  const int bh = p.batch * p.heads;
  mix_scan<<<dim3((most + 255) / 256, bh < 65535 ? bh : 65535, p.count), 256, 0, st>>>(p);
  return hipGetLastError();
}

hipError_t launch_mix_share(const MixShare& p, hipStream_t st) {
  int most = 0;
  for (int i = 0; i < p.count; ++i) most = p.one[i].dim > most ? p.one[i].dim : most;
  int64_t across = 1;
  while (4 * across < most) across *= 2;
  const int64_t want = (p.rows * p.kv_heads * across + 255) / 256;
  mix_share<<<dim3(static_cast<unsigned>(want < 65536 ? want : 65536), p.count), 256, 0, st>>>(p);
  return hipGetLastError();
}

hipError_t launch_mix_step(bool f32, const MixStep& p, hipStream_t st) {
  const dim3 grid(p.batch * p.heads, (p.dim_v + 4 * p.lanes - 1) / (4 * p.lanes));
  if (f32) mix_step<true><<<grid, 256, 0, st>>>(p);
  else mix_step<false><<<grid, 256, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace muon
