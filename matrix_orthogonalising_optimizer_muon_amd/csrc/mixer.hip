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
// A workgroup of four waves walks the chunks of one (batch, head), or of a segment of it, for a
// slice of dim_v columns. The state stays in its accumulators; only a rounded copy goes through
// LDS, as the operand of q Z. Products on 16 x 16 tiles, transposed (rows: s, dim_v or dim;
// columns: tokens), so that a lane's four results are neighbours along the axis that the next
// product sums over: the scores of a token become the operand of the product with v without
// leaving the lane, the state's copy and the output leave in 16 bytes.
#include "layer.hpp"
#include "mfma_util.hpp"

namespace muon {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));

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

// Which column row m of 16-row tile `t` stands for. 16-bit: tiles go in pairs that interleave
// by fours, so that a lane's results of both are eight neighbours (16 bytes).
template <bool F32>
__device__ __forceinline__ int col_of(int t, int m) {
  return F32 ? 16 * t + m : 32 * (t >> 1) + 8 * (m >> 2) + 4 * (t & 1) + (m & 3);
}

__device__ __forceinline__ u32x2 read_transposed(const __attribute__((address_space(3))) unsigned short* __restrict__ p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p));
}

// The fragment of tile t's columns (as rows) over tokens, from an array of tokens (rows of
// PITCH bytes). Tokens in the order the scores' results have: 16-bit step s: 32 s + 16 (e / 4) +
// 4 (l / 16) + e % 4 for e = 0..7; fp32: 16 s + 4 (l / 16) + e. BY_TILE: the fours of columns lie by tile.
template <bool F32, int PITCH, bool BY_TILE>
__device__ __forceinline__ u32x4 columns(const char* lds, int t, int s, int lane) {
  const int g = lane >> 4, i = lane & 15;
  u32x4 f;
  if constexpr (F32) {
    const char* p = lds + (16 * s + 4 * g) * PITCH + col_of<F32>(t, i) * 4;
#pragma unroll
    for (int r = 0; r < 4; ++r) f[r] = *reinterpret_cast<const unsigned int*>(p + r * PITCH);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // 16 lanes read four rows of four pieces; lane i receives column i of the 16
      const int c = BY_TILE ? 16 * t + 4 * (i & 3) : col_of<F32>(t, 4 * (i & 3));
      const char* p = lds + (32 * s + 16 * h + 4 * g + (i >> 2)) * PITCH + c * 2;
      const u32x2 r = read_transposed((const __attribute__((address_space(3))) unsigned short*)p);
      f[2 * h] = r[0];
      f[2 * h + 1] = r[1];
    }
  }
  return f;
}

// 16 bytes of a row from column c on.
template <bool F32>
__device__ __forceinline__ u32x4 load_whole(const char* row, int c) {
  if constexpr (F32) return *reinterpret_cast<const u32x4_a4*>(row + c * 4);
  else return *reinterpret_cast<const u32x4_a2*>(row + c * 2);
}
// The same with zeros behind its `dim` columns.
template <bool F32>
__device__ __forceinline__ u32x4 load_row(const char* row, int c, int dim) {
  constexpr int VEC = Type<F32>::VEC;
  if (c + VEC <= dim) return load_whole<F32>(row, c);
  u32x4 v{0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    if (c + e < dim) {
      if constexpr (F32) v[e] = *reinterpret_cast<const unsigned int*>(row + (c + e) * 4);
      else v[e / 2] |= static_cast<unsigned int>(*reinterpret_cast<const unsigned short*>(row + (c + e) * 2)) << (16 * (e & 1));
    }
  }
  return v;
}

// Waits for this workgroup's LDS traffic and its waves. The two kinds of waves below meet here from
// loops of their own, with the same number of turns.
__device__ __forceinline__ void meet() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
}

// Four waves keep the state (each dim / 4 of its rows, or half of rows and columns), with OUT four
// more make the outputs (16 of a chunk's tokens each): a SIMD then has one of either, whose matrix
// instructions, conversions and LDS reads fill each other's gaps. BUFS copies of a chunk's operands
// in LDS: with two the next chunk's are written while this one's are read.
template <bool F32, int DP, int NV, bool OUT>
__global__ __launch_bounds__(OUT ? 512 : 256, OUT ? 2 : 2) void mix_walk(const MixParams p) {
  constexpr int ES = Type<F32>::ES, VEC = Type<F32>::VEC, KF = Type<F32>::KF;
  constexpr int THREADS = OUT ? 512 : 256;
  constexpr int PB = DP * ES + 16, PC = NV * ES + (F32 ? 16 : 32);   // rows of LDS in bytes
  constexpr int WD = DP == 64 ? 2 : 4, WE = 4 / WD;            // waves over the state's rows and columns
  constexpr int MT = DP / WD / 16, NT = NV / WE / 16;          // its 16 x 16 tiles a wave
  constexpr int JS = C / KF;                                   // fragments over a chunk's tokens
  constexpr int DS = DP / KF;                                  // fragments over dim
  constexpr int LB = (C * DP / VEC + THREADS - 1) / THREADS, LC = (C * NV / VEC + THREADS - 1) / THREADS;  // loads a thread and chunk
  constexpr int TILES = NV / 16;
  constexpr int SET = C * PB + C * PC + (OUT ? NV * PB : 0);
  constexpr int BUFS = 2 * SET <= (OUT ? 160 : 80) * 1024 ? 2 : 1;
  static_assert(MT * WD * 16 == DP && NT * WE * 16 == NV, "whole tiles");
  __shared__ __attribute__((aligned(16))) char lds[BUFS * SET];

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

  // ---- b and c of a chunk: on their way in registers, then in LDS ----
  const char* rows_b = base(o.b);
  const char* rows_c = base(o.c) + e0 * ES;
  const int64_t sb = o.b.st * ES, sc = o.c.st * ES;
  u32x4 nb[LB], nc[LC];
  auto request = [&](int r0) {
    const bool inside = r0 + C <= live;
    if (inside && dim == DP) {
#pragma unroll
      for (int j = 0; j < LB; ++j) {
        const int x = j * THREADS + tid, row = x / (DP / VEC), c = x % (DP / VEC) * VEC;
        if (C * DP / VEC % THREADS == 0 || row < C) nb[j] = load_whole<F32>(rows_b + token(r0 + row) * sb, c);
      }
    } else {
#pragma unroll
      for (int j = 0; j < LB; ++j) {
        const int x = j * THREADS + tid, row = x / (DP / VEC), c = x % (DP / VEC) * VEC;
        nb[j] = u32x4{0, 0, 0, 0};
        if (row < C && r0 + row < live && c < dim) nb[j] = load_row<F32>(rows_b + token(r0 + row) * sb, c, dim);
      }
    }
    if (inside && cols == NV) {
#pragma unroll
      for (int j = 0; j < LC; ++j) {
        const int x = j * THREADS + tid, row = x / (NV / VEC), c = x % (NV / VEC) * VEC;
        if (C * NV / VEC % THREADS == 0 || row < C) nc[j] = load_whole<F32>(rows_c + token(r0 + row) * sc, c);
      }
    } else {
#pragma unroll
      for (int j = 0; j < LC; ++j) {
        const int x = j * THREADS + tid, row = x / (NV / VEC), c = x % (NV / VEC) * VEC;
        nc[j] = u32x4{0, 0, 0, 0};
        if (row < C && r0 + row < live && c < cols) nc[j] = load_row<F32>(rows_c + token(r0 + row) * sc, c, cols);
      }
    }
  };
  auto keep = [&](char* set) {
#pragma unroll
    for (int j = 0; j < LB; ++j) {
      const int x = j * THREADS + tid;
      if (C * DP / VEC % THREADS == 0 || x < C * DP / VEC)
        *reinterpret_cast<u32x4*>(set + x / (DP / VEC) * PB + x % (DP / VEC) * 16) = nb[j];
    }
#pragma unroll
    for (int j = 0; j < LC; ++j) {
      const int x = j * THREADS + tid, ch = x % (NV / VEC);
      char* row = set + C * PB + x / (NV / VEC) * PC;
      if (C * NV / VEC % THREADS == 0 || x < C * NV / VEC) {
        if constexpr (F32) {
          *reinterpret_cast<u32x4*>(row + ch * 16) = nc[j];
        } else {
          // columns by tile: of 32, the fours of the even tile first (its transpose reads then take 32 bytes a row)
          *reinterpret_cast<u32x2*>(row + (ch >> 2) * 64 + (ch & 3) * 8) = u32x2{nc[j][0], nc[j][1]};
          *reinterpret_cast<u32x2*>(row + (ch >> 2) * 64 + (ch & 3) * 8 + 32) = u32x2{nc[j][2], nc[j][3]};
        }
      }
    }
  };

  const bool carried = o.z_in && (p.z_in_per_segment || seg == 0);
  if (begin < live) request(begin);

  if (!OUT || wave >= 4) {
    // ---- the state: rows d = dbase + col_of(mt, .), columns e = col_of(we NT + nt, .) ----
    const int own = wave & 3, wd = own % WD, we = own / WD;
    const int dbase = wd * (DP / WD);
    f32x4 z[MT][NT];
    {
      const float* src = nullptr;
      if (carried) src = o.z_in + (p.z_in_per_segment ? static_cast<int64_t>(bh) * p.segments + seg : bh) * dim * dim_v;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int e = col_of<F32>(we * NT + nt, l16);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int d = dbase + col_of<F32>(mt, 4 * g + r);
            z[mt][nt][r] = src && d < dim && e < cols ? src[d * o.z_row + (e0 + e) * o.z_col] : 0.0f;
          }
        }
    }
    // its copy for the outputs, dim_v (by tile) x dim. 16-bit: rounded to bf16, as the operand of q Z, like the
    // scores as that of the product with v
    auto show = [&](char* set) {
      if constexpr (OUT) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          char* row = set + C * (PB + PC) + (16 * (we * NT + nt) + l16) * PB + dbase * ES;
          if constexpr (F32) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              *reinterpret_cast<u32x4*>(row + (16 * mt + 4 * g) * 4) = __builtin_bit_cast(u32x4, z[mt][nt]);
          } else {
#pragma unroll
            for (int mt = 0; mt < MT; mt += 2)
              *reinterpret_cast<u32x4*>(row + (16 * mt + 8 * g) * 2) =
                  u32x4{pack(z[mt][nt][0], z[mt][nt][1]), pack(z[mt][nt][2], z[mt][nt][3]),
                        pack(z[mt + 1][nt][0], z[mt + 1][nt][1]), pack(z[mt + 1][nt][2], z[mt + 1][nt][3])};
          }
        }
      }
    };
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
    float over = __builtin_amdgcn_exp2f(g2 * C);

    if (begin < live) {
      keep(lds);
      show(lds);
    }
    int buf = 0;
    for (int r0 = begin; r0 < live; r0 += C) {
      const char* set = lds + buf * SET;
      meet();
      const bool more = r0 + C < live;
      if (more) request(r0 + C);
      const int rows = min(live - r0, C);
      if (rows < C) {
        weigh(rows);
        over = __builtin_amdgcn_exp2f(g2 * rows);
      }
      // weighted b of this wave's rows. 16-bit: as three parts whose sum has the product's 24
      // bits, so that the state is the sum of unrounded terms
      constexpr int PARTS = F32 ? 1 : 3;
      u32x4 kf[PARTS][MT][JS];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int s = 0; s < JS; ++s) {
          const u32x4 f = columns<F32, PB, false>(set + dbase * ES, mt, s, lane);
          if constexpr (F32) {
#pragma unroll
            for (int e = 0; e < 4; ++e) kf[0][mt][s][e] = __float_as_uint(__uint_as_float(f[e]) * weight[s][e]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float lo = __uint_as_float(f[e] << 16) * weight[s][2 * e];
              float hi = __uint_as_float(f[e] & 0xFFFF0000u) * weight[s][2 * e + 1];
#pragma unroll
              for (int q = 0; q < PARTS; ++q) {
                const unsigned int w = pack(lo, hi);
                kf[q][mt][s][e] = w;
                lo -= __uint_as_float(w << 16);
                hi -= __uint_as_float(w & 0xFFFF0000u);
              }
            }
          }
        }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        u32x4 v[JS];
#pragma unroll
        for (int s = 0; s < JS; ++s) v[s] = columns<F32, PC, true>(set + C * PB, we * NT + nt, s, lane);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          z[mt][nt] *= over;
#pragma unroll
          for (int s = 0; s < JS; ++s)
#pragma unroll
            for (int q = 0; q < PARTS; ++q) mma<F32>(z[mt][nt], kf[q][mt][s], v[s]);
        }
      }
      if (more) {
        if constexpr (BUFS == 1) meet();
        buf = BUFS == 2 ? buf ^ 1 : 0;
        keep(lds + buf * SET);
        show(lds + buf * SET);
      }
    }

    if (o.z_out && (p.z_out_per_segment || seg == (n > 0 ? (n - 1) / p.segment : 0))) {
      float* dst = o.z_out + (p.z_out_per_segment ? static_cast<int64_t>(bh) * p.segments + seg : bh) * dim * dim_v;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int e = col_of<F32>(we * NT + nt, l16);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int d = dbase + col_of<F32>(mt, 4 * g + r);
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
    u32x4 na[DS];
    auto request_a = [&](int r0) {
      const char* row = rows_a + token(r0 + i_tok) * sa;
      if (r0 + C <= live && dim == DP) {
#pragma unroll
        for (int s = 0; s < DS; ++s) na[s] = load_whole<F32>(row, KF * s + VEC * g);
      } else {
#pragma unroll
        for (int s = 0; s < DS; ++s) {
          const int c = KF * s + VEC * g;
          na[s] = u32x4{0, 0, 0, 0};
          if (r0 + i_tok < live && c < dim) na[s] = load_row<F32>(row, c, dim);
        }
      }
    };
    float within[4][4];                                         // e^{g (i - s)} of the scores' tiles
#pragma unroll
    for (int jt = 0; jt < 4; ++jt)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        within[jt][r] = __builtin_amdgcn_exp2f(g2 * max(i_tok - (16 * jt + 4 * g + r), 0)) * o.p_scale;
    const float reach = __builtin_amdgcn_exp2f(g2 * (i_tok + off)) * o.o_scale;
    const int64_t o_row = static_cast<int64_t>(p.heads) * dim_v;   // elements from token to token of the output
    const int64_t o_at = (static_cast<int64_t>(batch) * p.tokens * p.heads + head) * dim_v + e0;

    if (begin < live) {
      request_a(begin);
      keep(lds);
    }
    int buf = 0;
    for (int r0 = begin; r0 < live; r0 += C) {
      const char* set = lds + buf * SET;
      meet();
      const bool more = r0 + C < live;
      u32x4 a[DS];
#pragma unroll
      for (int s = 0; s < DS; ++s) a[s] = na[s];
      if (more) {
        request(r0 + C);
        request_a(r0 + C);
      }
      // scores, transposed: rows s (the chunk's tokens up to its own), columns this wave's tokens
      u32x4 score[JS];
      {
        f32x4 sc4[4];
#pragma unroll
        for (int jt = 0; jt < 4; ++jt) {
          sc4[jt] = f32x4{0, 0, 0, 0};
          if (jt <= wave) {
#pragma unroll
            for (int s = 0; s < DS; ++s) {
              const u32x4 k = *reinterpret_cast<const u32x4*>(set + (16 * jt + l16) * PB + (KF * s + VEC * g) * ES);
              mma<F32>(sc4[jt], k, a[s]);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) sc4[jt][r] *= within[jt][r];
            if (jt == wave) {
#pragma unroll
              for (int r = 0; r < 4; ++r) sc4[jt][r] = 4 * g + r <= l16 ? sc4[jt][r] : 0.0f;
            }
          }
        }
#pragma unroll
        for (int s = 0; s < JS; ++s) {
          if constexpr (F32) score[s] = __builtin_bit_cast(u32x4, sc4[s]);
          else
            score[s] = u32x4{pack(sc4[2 * s][0], sc4[2 * s][1]), pack(sc4[2 * s][2], sc4[2 * s][3]),
                             pack(sc4[2 * s + 1][0], sc4[2 * s + 1][1]), pack(sc4[2 * s + 1][2], sc4[2 * s + 1][3])};
        }
      }
      const bool have = carried || r0 > begin;
      const bool mine = o.out && r0 + i_tok < live;
      const int64_t o_tok = o_at + token(r0 + i_tok) * o_row;
      f32x4 acc[2];
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        f32x4 x{0, 0, 0, 0};
        if (have) {
#pragma unroll
          for (int s = 0; s < DS; ++s) {
            const u32x4 k = *reinterpret_cast<const u32x4*>(set + C * (PB + PC) + (16 * t + l16) * PB + (KF * s + VEC * g) * ES);
            mma<F32>(x, k, a[s]);
          }
          x *= reach;
        }
#pragma unroll
        for (int s = 0; s < JS; ++s)
          if (KF * s <= 16 * wave) mma<F32>(x, columns<F32, PC, true>(set + C * PB, t, s, lane), score[s]);
        acc[t & 1] = x;
        // lane: token i_tok, columns of the tile (pair) 16 g .. or 32 .. + 8 g ..
        if constexpr (F32) {
          if (mine) {
            float* out = static_cast<float*>(o.out) + o_tok + 16 * t + 4 * g;
            const int left = cols - (16 * t + 4 * g);
            if (left >= 4) *reinterpret_cast<u32x4_a4*>(out) = __builtin_bit_cast(u32x4, x);
            else
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (r < left) out[r] = x[r];
          }
        } else if (t & 1) {
          const int c = 32 * (t >> 1) + 8 * g, left = cols - c;
          if (mine && o.out_f32) {
            float* out = static_cast<float*>(o.out) + o_tok + c;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (left >= 4 * h + 4) *reinterpret_cast<u32x4_a4*>(out + 4 * h) = __builtin_bit_cast(u32x4, acc[h]);
              else
#pragma unroll
                for (int r = 0; r < 4; ++r)
                  if (4 * h + r < left) out[4 * h + r] = acc[h][r];
            }
          } else if (mine) {
            unsigned short* out = static_cast<unsigned short*>(o.out) + o_tok + c;
            const u32x4 w{pack(acc[0][0], acc[0][1]), pack(acc[0][2], acc[0][3]), pack(acc[1][0], acc[1][1]),
                          pack(acc[1][2], acc[1][3])};
            if (left >= 8) *reinterpret_cast<u32x4_a2*>(out) = w;
            else
#pragma unroll
              for (int r = 0; r < 8; ++r)
                if (r < left) out[r] = static_cast<unsigned short>(w[r / 2] >> (16 * (r & 1)));
          }
        }
      }
      if (more) {
        if constexpr (BUFS == 1) meet();
        buf = BUFS == 2 ? buf ^ 1 : 0;
        keep(lds + buf * SET);
      }
    }
    // rows behind the last token: zeros
    const int first = max(live, begin);
    const int64_t count = o.out ? static_cast<int64_t>(end - first) * cols : 0;
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
    float g2 = p.log_decay[bh % p.heads] * kLog2e;
    g2 = g2 < -1e30f ? -1e30f : g2;
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
        s = __builtin_amdgcn_exp2f(g2 * len) * s + u[k];
      }
    }
  }
}

// Gradients of shared heads: the group's fp32 partial sums in head order, rounded once.
__global__ __launch_bounds__(256) void mix_share(const MixShare p) {
  const auto o = p.one[blockIdx.y];
  const int64_t n = p.rows * p.kv_heads * o.dim;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t row = i / o.dim, d = i % o.dim;
    const float* q = o.part + row * p.group * o.dim + d;
    float s = q[0];
    for (int k = 1; k < p.group; ++k) s += q[static_cast<int64_t>(k) * o.dim];
    if (p.bf16) static_cast<unsigned short*>(o.out)[i] = to_bf16(s);
    else static_cast<float*>(o.out)[i] = s;
  }
}

// One token: S' = e^g S + k^T v, o = scale q S'. Bound by the state's traffic, read and written
// once. A workgroup takes `lanes` threads of four columns across and 256 / lanes rows at a time;
// their sums are joined in LDS in row order.
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
  const float decay = __builtin_amdgcn_exp2f(p.log_decay[h] * kLog2e);
  const int left = p.dim_v - e;
  f32x4 v{0, 0, 0, 0}, acc{0, 0, 0, 0};
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (r < left) v[r] = load_one<F32>(p.v, b * p.v_sb + (h / p.group) * p.v_sh + e + r);
  __syncthreads();
  const int64_t at = static_cast<int64_t>(bh) * p.dim * p.dim_v + e;
  if (left >= 4) {
#pragma unroll 4
    for (int d = down; d < p.dim; d += rows) {
      const int64_t x = at + static_cast<int64_t>(d) * p.dim_v;
      f32x4 s = __builtin_bit_cast(f32x4, static_cast<u32x4>(*reinterpret_cast<const u32x4_a4*>(p.z_in + x)));
      s = s * decay + v * qk[1][d];
      *reinterpret_cast<u32x4_a4*>(p.z_out + x) = __builtin_bit_cast(u32x4, s);
      acc += s * qk[0][d];
    }
  } else {
    for (int d = down; d < p.dim; d += rows)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r < left) {
          const int64_t x = at + static_cast<int64_t>(d) * p.dim_v + r;
          const float s = p.z_in[x] * decay + v[r] * qk[1][d];
          p.z_out[x] = s;
          acc[r] += s * qk[0][d];
        }
  }
  sums[tid] = acc;
  __syncthreads();
  if (down == 0) {
    for (int k = 1; k < rows; ++k) acc += sums[k * p.lanes + across];
    const int64_t x = static_cast<int64_t>(bh) * p.dim_v + e;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (r < left) {
        if constexpr (F32) static_cast<float*>(p.out)[x + r] = acc[r];
        else static_cast<unsigned short*>(p.out)[x + r] = to_bf16(acc[r]);
      }
  }
}

template <bool F32, int DP, int NV>
hipError_t walk(bool out, const MixParams& p, int64_t groups, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(groups));
  if (out) mix_walk<F32, DP, NV, true><<<grid, 512, 0, st>>>(p);
  else mix_walk<F32, DP, NV, false><<<grid, 256, 0, st>>>(p);
  return hipGetLastError();
}
template <bool F32>
hipError_t walk(MixTile t, bool out, const MixParams& p, int64_t groups, hipStream_t st) {
  if (t.dim == 64) return t.dim_v == 64 ? walk<F32, 64, 64>(out, p, groups, st) : walk<F32, 64, 32>(out, p, groups, st);
  if (t.dim == 128)
    return t.dim_v == 128 ? walk<F32, 128, 128>(out, p, groups, st)
           : t.dim_v == 64 ? walk<F32, 128, 64>(out, p, groups, st) : walk<F32, 128, 32>(out, p, groups, st);
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
  int64_t most = 0;
  for (int i = 0; i < p.count; ++i) most = p.one[i].dim > most ? p.one[i].dim : most;
  const int64_t want = (p.rows * p.kv_heads * most + 255) / 256;
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
