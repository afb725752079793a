// Device helpers of the training operators' kernels (ffn.hip, losses.hip): vector types, LDS
// chunk swizzle, counter waits and the direct global -> LDS loads of gfx950. gemm.hip keeps
// its own copies: the HBM traffic records of its profiles are tied to that file's contents.
#pragma once

#include "internal.hpp"

namespace muon {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// XOR swizzle of LDS rows of CH 16-byte chunks, so that fragment reads of 32 consecutive
// rows spread over all banks (CH = 8: 128-byte rows; CH = 4: 64-byte rows, two per 128 bytes,
// where rows 2t and 2t+1 share the XOR term so that 8 consecutive rows read at one logical
// chunk still cover all eight 16-byte positions of a 128-byte span).
template <int CH>
__device__ __forceinline__ int swz_bits(int row) {
  static_assert(CH == 8 || CH == 4, "chunks per row");
  return CH == 8 ? ((row ^ (row >> 3)) & 7) : ((row >> 1) & 3);
}
template <int CH>
__device__ __forceinline__ int swz_ch(int row, int chunk) {
  return row * CH + (chunk ^ swz_bits<CH>(row));
}

// s_waitcnt with only the vector-memory counter constrained (gfx9 encoding: vmcnt in bits
// 3:0 and 15:14; expcnt 6:4 and lgkmcnt 11:8 left at their maxima).
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
// Buffer resource over `bytes` bytes from `base` (raw buffer: no stride, no format
// conversion; accesses at or past `bytes` return zero instead of faulting).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, static_cast<int>(bytes), 0x00020000);
}
// 16 bytes per lane from the buffer at voff + soff into LDS: lane l writes bytes
// [16 l, 16 l + 16) of the instruction's window at lds_dst (the M0 base).
__device__ __forceinline__ void buf_load_lds(__amdgpu_buffer_rsrc_t r, void* lds_dst, uint32_t voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds_dst, 16, voff, soff, 0, 0);
}

// wait_vmcnt, and every LDS access of this wave returned (lgkmcnt 0).
template <int N>
__device__ __forceinline__ void wait_vmcnt_lgkm0() {
  static_assert(N >= 0 && N < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

}  // namespace
}  // namespace muon
