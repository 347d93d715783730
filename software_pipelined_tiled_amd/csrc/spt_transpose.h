// Operand tiles that are contiguous in the output's direction, turned on the way from LDS to registers.
//
// Such a tile is 64 rows of c (the summed index) by R columns. ds_read_b64_tr_b16 makes a matrix operand
// of it: in each quarter-wave, lane p supplies the address of columns 4 (p % 4) .. +3 of row p / 4 and
// receives column p of the four rows, so two reads give a lane eight c of one column.
//
// Row c holds R / 8 chunks of 16 bytes; chunk q sits at chunk q XOR 2 tr_swz(c). The LDS serves 32 lanes a
// cycle from 64 banks: four rows of two neighbouring chunks for each of two quarter-waves, eight rows of
// c apart. The XOR spreads those eight 32-byte pieces over the 256 bytes the banks span (measured with
// SQ_LDS_BANK_CONFLICT: none; with the quarter-waves' rows alike, half of the read cycles).
#pragma once

#include "spt_device.h"

namespace spt {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4_t;

template <int R>
__device__ __forceinline__ int tr_swz(int c) {
  static_assert(R == 64 || R >= 128, "rows of 128 bytes, or 256 and more");
  return R == 64 ? ((c >> 1) & 1) | ((c >> 2) & 2) : (c & 3) | ((c >> 1) & 4);
}

// LDS byte offset of the 32 bytes that hold columns 16 u .. 16 u + 15 of row c
template <int R>
__device__ __forceinline__ int tr_offset(int c, int u) {
  return c * (2 * R) + ((u ^ tr_swz<R>(c)) << 5);
}

// The fragment whose lanes' addresses are p, for c rows 0 .. 3 and 4 .. 7 of the lane's eight; ROW: bytes of
// a row of c.
template <int ROW>
__device__ __forceinline__ u32x4 tr_frag(lds_void_t* p) {
  const uint64_t a = __builtin_bit_cast(uint64_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)p));
  const uint64_t b = __builtin_bit_cast(
      uint64_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)((__attribute__((address_space(3))) char*)p + 4 * ROW)));
  return u32x4{(unsigned)a, (unsigned)(a >> 32), (unsigned)b, (unsigned)(b >> 32)};
}
template <int ROW>
__device__ __forceinline__ u32x4 tr_frag(const char* p) {
  return tr_frag<ROW>((lds_void_t*)(const lds_void_t*)p);
}

// v ^ c (c wave-uniform), and (v ^ c) + d, computed where they are written: the compiler may not keep one
// register per c instead.
__device__ __forceinline__ unsigned xor_in_place(unsigned v, unsigned c) {
  unsigned r;
  asm volatile("v_xor_b32 %0, %1, %2" : "=v"(r) : "s"(c), "v"(v));
  return r;
}
__device__ __forceinline__ unsigned xor_add_in_place(unsigned v, unsigned c, unsigned d) {
  unsigned r;
  asm volatile("v_xad_u32 %0, %1, %2, %3" : "=v"(r) : "v"(v), "s"(c), "v"(d));
  return r;
}

// With such a tile as the matrix instruction's first operand, lane l holds columns 4 (l / 16) .. +3 of each
// 16-column block, row l % 16. Exchanging the odd quarter-waves of one block with the even ones of the next
// gives every lane eight consecutive columns: 16 ((l / 16) % 2) + 8 (l / 32) of the pair's 32.
__device__ __forceinline__ void pair_columns(const f32x4& lo, const f32x4& hi, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float l = lo[e], h = hi[e];
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, l), __builtin_bit_cast(unsigned, h),
                                                    false, false);
    const unsigned a = r[0], b = r[1];
    v[e] = __builtin_bit_cast(float, a);
    v[4 + e] = __builtin_bit_cast(float, b);
  }
}
__device__ __forceinline__ int pair_column(int lane) { return 16 * ((lane >> 4) & 1) + 8 * (lane >> 5); }

// Four consecutive fp32 outputs at row m (relative to the descriptor's first), column n. Lanes whose
// columns follow each other write 64 or 256 contiguous bytes per store; the eight columns a lane holds for a
// 16-bit output would be two stores with 16-byte gaps, at half the rate. EDGE as in store8.
template <bool EDGE>
__device__ __forceinline__ void store4_f32(const f32x4& v, __amdgpu_buffer_rsrc_t rc, int m, int rows_left, int n, int N,
                                           int ldc) {
  if (EDGE && (m >= rows_left || n >= N)) return;
  const unsigned off = (unsigned)(m * ldc + n) * 4u;
  if (!EDGE || n + 4 <= N) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rc, off, 0, 0);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float f = v[e];
      if (n + e < N) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, f), rc, off + 4u * e, 0, 0);
    }
  }
}

}  // namespace spt
