// Device helpers of the microscaled operators and the norm: rows in pieces of eight values, conversions to and from
// the formats, the scaled matrix instruction.
#pragma once

#include "spt_device.h"
#include "spt_mx.h"

namespace spt {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x2 __attribute__((ext_vector_type(2)));

constexpr int kTypeSize[3] = {2, 2, 4};  // f16, bf16, f32

// 16 bytes at any element's alignment: the memory path takes dwords off their own size (1003 rows of 4097 fp32 through the
// norm and its gradients: 25 us, 86 with an element at a time).
typedef unsigned u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef unsigned u32_any __attribute__((aligned(2)));

// Eight values of type T as they lie in memory.
template <int T>
struct Raw8 {
  u32x4 q[T == 2 ? 2 : 1];
};

// Eight values at `p`, of which `left` are there; the others become zeros. A row's end goes straight to its words, in 16 bits by pieces
// of four, two and one (5000 rows of 8190 fp16 to 4 bits: 20 us, 40 with 16-bit values put together one by one).
template <int T>
__device__ __forceinline__ Raw8<T> load_raw(const char* p, int left) {
  Raw8<T> r;
  if (left >= 8) {
    r.q[0] = *(const u32x4_any*)p;
    if constexpr (T == 2) r.q[1] = *(const u32x4_any*)(p + 16);
    return r;
  }
  r.q[0] = u32x4{0, 0, 0, 0};
  if constexpr (T == 2) {
    r.q[1] = r.q[0];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) r.q[e >> 2][e & 3] = ((const unsigned*)p)[e];
  } else if (left > 0) {
    const int tail = __builtin_amdgcn_readfirstlane(left);  // a row's last lane: the same of every row here
    auto two_and_one = [&](auto at_c) SPT_INLINE {
      constexpr int at = decltype(at_c)::value;
      if (tail & 2) {
        r.q[0][at] = *(const u32_any*)(p + at * 4);
        if (tail & 1) r.q[0][at + 1] = *(const unsigned short*)(p + at * 4 + 4);
      } else if (tail & 1) {
        r.q[0][at] = *(const unsigned short*)(p + at * 4);
      }
    };
    if (tail & 4) {
      const u32x2 v = *(const u32x2_any*)p;
      r.q[0][0] = v[0];
      r.q[0][1] = v[1];
      two_and_one(std::integral_constant<int, 2>{});
    } else {
      two_and_one(std::integral_constant<int, 0>{});
    }
  }
  return r;
}

// Eight values of a row of n from `col` on, for a load that goes out ahead of its use: the row's end is loaded as its last eight values,
// and `settle` shifts them into place where they are used. With load_raw's branches the compiler waits for the load, or
// moves the values' conversion, up to the load (5000 rows of 8190 bf16 through the norm with its residual: 63 us, 91; 8191 rows of
// 8192 fp16: 104, 124).
template <int T>
__device__ __forceinline__ Raw8<T> load_ahead(const char* row, int col, int n) {
  constexpr int ES = kTypeSize[T];
  Raw8<T> r;
  if (n < 8) {
    r = load_raw<T>(row + (unsigned)(col * ES), n - col);
#pragma unroll
    for (int i = 0; i < (T == 2 ? 8 : 4); ++i) r.q[i / 4][i % 4] = opaque_u32(r.q[i / 4][i % 4]);  // the conversion stays behind it here too
    return r;
  }
  const char* p = row + (unsigned)((col < n - 8 ? col : n - 8) * ES);
  r.q[0] = *(const u32x4_any*)p;
  if constexpr (T == 2) r.q[1] = *(const u32x4_any*)(p + 16);
  return r;
}
template <int T>
__device__ __forceinline__ void settle(Raw8<T>& r, int col, int n) {
  const int miss = col - (n - 8);
  if (miss <= 0 || n < 8) return;
  constexpr int N = T == 2 ? 8 : 4;
  unsigned w[N];
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = miss < 8 ? r.q[i / 4][i % 4] : 0u;
#pragma unroll
  for (int d = N / 2; d >= 1; d /= 2) {  // whole words
    const bool move = (miss & (T == 2 ? d : 2 * d)) != 0;
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = move ? (i + d < N ? w[i + d] : 0u) : w[i];
  }
  if constexpr (T != 2) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = (miss & 1) ? w[i] >> 16 | (i + 1 < N ? w[i + 1] << 16 : 0u) : w[i];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) r.q[i / 4][i % 4] = w[i];
}

template <int T>
__device__ __forceinline__ void unpack(const Raw8<T>& r, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (T == 2) {
      const unsigned word = r.q[e >> 2][e & 3];  // (a bit_cast of the element itself would take the vector's first)
      v[e] = __builtin_bit_cast(float, word);
    } else if constexpr (T == 1) v[e] = __builtin_bit_cast(float, (e & 1) ? r.q[0][e >> 1] & 0xFFFF0000u : r.q[0][e >> 1] << 16);
    else v[e] = (float)__builtin_bit_cast(_Float16, (unsigned short)(r.q[0][e >> 1] >> (16 * (e & 1))));
  }
}

// Eight floats rounded to type T.
template <int T>
__device__ __forceinline__ Raw8<T> pack(const float (&v)[8]) {
  Raw8<T> r;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (T == 2) {
      r.q[0][e] = __builtin_bit_cast(unsigned, v[e]);
      r.q[1][e] = __builtin_bit_cast(unsigned, v[4 + e]);
    } else {
      r.q[0][e] = T == 1 ? pack_bf16(v[2 * e], v[2 * e + 1]) : pack_f16(v[2 * e], v[2 * e + 1]);
    }
  }
  return r;
}

template <int T>
__device__ __forceinline__ void put_raw(char* p, int left, const Raw8<T>& r) {
  if (left >= 8) {
    *(u32x4_any*)p = r.q[0];
    if constexpr (T == 2) *(u32x4_any*)(p + 16) = r.q[1];
    return;
  }
  if (left <= 0) return;
  const int tail = __builtin_amdgcn_readfirstlane(left);
  auto two_and_one = [&](auto at_c) SPT_INLINE {
    constexpr int at = decltype(at_c)::value;
    auto w = [&](int i) SPT_INLINE { return r.q[(at + i) / 4][(at + i) % 4]; };
    char* q = p + at * 4;
    if constexpr (T == 2) {
      if (tail & 2) *(u32x2_any*)q = u32x2{w(0), w(1)};
      if (tail & 1) *(unsigned*)(q + (tail & 2) * 4) = tail & 2 ? w(2) : w(0);
    } else {
      if (tail & 2) *(u32_any*)q = w(0);
      if (tail & 1) *(unsigned short*)(q + (tail & 2) * 2) = (unsigned short)(tail & 2 ? w(1) : w(0));
    }
  };
  if (tail & 4) {
    if constexpr (T == 2) *(u32x4_any*)p = r.q[0];
    else *(u32x2_any*)p = u32x2{r.q[0][0], r.q[0][1]};
    two_and_one(std::integral_constant<int, T == 2 ? 4 : 2>{});
  } else {
    two_and_one(std::integral_constant<int, 0>{});
  }
}

template <int T>
__device__ __forceinline__ void load8(const char* p, int left, float (&v)[8]) {
  unpack<T>(load_raw<T>(p, left), v);
}
template <int T>
__device__ __forceinline__ void put8(char* p, int left, const float (&v)[8]) {
  put_raw<T>(p, left, pack<T>(v));
}

// Eight values of any type (a weight's): the type is the launch's, so the branch is the same for all lanes.
__device__ __forceinline__ void load8_any(const char* p, int type, int at, int left, float (&v)[8]) {
  if (type == 2) load8<2>(p + (int64_t)at * 4, left, v);
  else if (type == 1) load8<1>(p + (int64_t)at * 2, left, v);
  else load8<0>(p + (int64_t)at * 2, left, v);
}

// ------------------------------------------------------------------------------ formats
// A block's scale byte from eight values of each of its four lanes: the exponent of the largest magnitude less the
// format's largest one; 255 with an infinity or NaN among them, whose bits compare as larger than any number's.
template <int BITS>
__device__ __forceinline__ unsigned mx_scale_of(const float (&v)[8]) {
  unsigned m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const unsigned u = __builtin_bit_cast(unsigned, v[e]) & 0x7FFFFFFFu;
    m = u > m ? u : m;
  }
  const unsigned a = (unsigned)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true);  // quad lanes 1 0 3 2
  m = a > m ? a : m;
  const unsigned b = (unsigned)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true);  // quad lanes 2 3 0 1
  m = b > m ? b : m;
  const int field = (int)(m >> 23), s = field - (BITS == 4 ? 2 : 8);
  return field == 255 ? 255u : (unsigned)(s < 0 ? 0 : s);
}

// 2^(s - 127) for a byte s below 255.
__device__ __forceinline__ float mx_scale(unsigned s) { return __builtin_bit_cast(float, s ? s << 23 : 0x00400000u); }

// Eight values as codes, in 4 bytes (bits 4: the first word) or 8. The conversions divide by the scale and round to
// nearest, ties to even; the 4-bit one saturates, the 8-bit one does not, so its input is held to 448 scales before.
template <int BITS>
__device__ __forceinline__ u32x2 mx_codes(const float (&v)[8], unsigned s) {
  if (s == 255) return u32x2{0, 0};
  const float f = mx_scale(s);
  if constexpr (BITS == 4) {
    unsigned q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], f, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], f, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], f, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], f, 3);
    return u32x2{q, 0};
  } else {
    const float top = 448.f * f;
    float c[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = __builtin_amdgcn_fmed3f(v[e], -top, top);
    u32x2 r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      s16x2 p = {0, 0};
      p = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(p, c[4 * h], c[4 * h + 1], f, false);
      p = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(p, c[4 * h + 2], c[4 * h + 3], f, true);
      r[h] = __builtin_bit_cast(unsigned, p);
    }
    return r;
  }
}

// The eight values of codes; scale byte 255 makes them NaN. Unscaled values are exact, and so is ldexp up to fp32's own
// rounding of what lies below its normal numbers.
template <int BITS>
__device__ __forceinline__ void mx_values(u32x2 q, unsigned s, float (&v)[8]) {
  if constexpr (BITS == 4) {
    static_for<4>([&](auto i_c) SPT_INLINE {
      constexpr int i = decltype(i_c)::value;
      const f32x2 p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[0], 1.f, i);
      v[2 * i] = p[0];
      v[2 * i + 1] = p[1];
    });
  } else {
    static_for<4>([&](auto i_c) SPT_INLINE {
      constexpr int i = decltype(i_c)::value;
      const f32x2 p = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[i >> 1], (i & 1) != 0);
      v[2 * i] = p[0];
      v[2 * i + 1] = p[1];
    });
  }
  const float nan = __builtin_bit_cast(float, 0x7FC00000u);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = s == 255 ? nan : __builtin_ldexpf(v[e], (int)s - 127);
}

// ------------------------------------------------------------------------------ matrix instructions
// D[i][j] += sum over 128 k of X[i][k] Y[j][k], 16 x 16, each operand's 32-blocks scaled. Lane l supplies row l mod 16.
// In 4 bits its 16 bytes are block l / 16; in 8 bits its first 16 bytes are k = 16 (l / 16) .. +15 and the others 64
// further on. Byte SX (SY) of its scale word belongs to block l / 16 in both. It holds D[4 (l / 16) + e][l mod 16].
template <int FX, int FY, int SX, int SY>
__device__ __forceinline__ f32x4 mfma_mx(i32x8 x, i32x8 y, f32x4 c, unsigned sx, unsigned sy) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, FX == 8 ? 0 : 4, FY == 8 ? 0 : 4, SX, (int)sx, SY, (int)sy);
}

template <int F>
__device__ __forceinline__ i32x8 mx_operand(u32x4 lo, u32x4 hi) {
  if constexpr (F == 8) return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  else return __builtin_shufflevector(__builtin_bit_cast(__attribute__((ext_vector_type(4))) int, lo), __builtin_bit_cast(__attribute__((ext_vector_type(4))) int, lo), 0, 1, 2, 3, -1, -1, -1, -1);
}

// Eight of a lane's 32 values (part P) of one block as bf16, scaled: in 8 bits two words of `lo` and `hi`, in 4 bits word P of
// `lo`.
template <int F, int P>
__device__ __forceinline__ u32x4 mx_bf16(u32x4 lo, u32x4 hi, unsigned byte) {
  const float f = __builtin_bit_cast(float, byte << 23);  // the conversions take its exponent alone: 0 is 2^-127, 255 NaN
  u32x4 r;
  if constexpr (F == 8) {
    const unsigned w0 = P < 2 ? lo[2 * P % 4] : hi[2 * P % 4], w1 = P < 2 ? lo[2 * P % 4 + 1] : hi[2 * P % 4 + 1];
    r[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, f, false));
    r[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, f, true));
    r[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, f, false));
    r[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, f, true));
  } else {
    const unsigned w = lo[P];
    r[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 0));
    r[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 1));
    r[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 2));
    r[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 3));
  }
  return r;
}

// ------------------------------------------------------------------------------ products through bf16 at any scale
// A value times its scale is a bf16 number while the scale byte is in 10 .. 246 (2^-9 2^-117 is the smallest normal one, 448 2^119 is
// finite). Blocks beyond that are far, and k-steps with one take mx_far_products.

// Of words of four scale bytes: whether one is outside 64 .. 191, whose two highest bits are alike. OR a byte that nobody reads with 0x7F.
__device__ __forceinline__ bool mx_wide(unsigned wa, unsigned wb) { return (~((wa ^ (wa << 1)) & (wb ^ (wb << 1))) & 0x80808080u) != 0; }

// 0: near (NaN is), 1: low, 2: high.
__device__ __forceinline__ int mx_reach(unsigned byte) { return byte < 10 ? 1 : byte > 246 && byte < 255 ? 2 : 0; }

// The values of fragment `f` in a lane that are not zero, as bits.
template <int F, int N>
__device__ __forceinline__ unsigned mx_numbers(const u32x4 (&x)[N][F / 4], int f) {
  unsigned codes = 0;
#pragma unroll
  for (int h = 0; h < F / 4; ++h) codes |= x[f][h][0] | x[f][h][1] | x[f][h][2] | x[f][h][3];
  return codes & (F == 8 ? 0x7F7F7F7Fu : 0x77777777u);
}

// Nonzero if one of a lane's fragments (N of them, bytes of `w`) has a far scale and a value that is not zero.
template <int F, int N>
__device__ __forceinline__ unsigned mx_far(const u32x4 (&x)[N][F / 4], unsigned w) {
  unsigned any = 0;
  static_for<N>([&](auto f_c) SPT_INLINE {
    constexpr int f = decltype(f_c)::value;
    const unsigned from = ((w >> (8 * f)) & 255u) - 10;  // 0 .. 236: near, 245: NaN
    any |= (from > 236) & (from != 245) ? mx_numbers<F, N>(x, f) : 0u;
  });
  return any;
}

// The reaches of the wave's blocks that are not zero, one bit each; near always.
template <int F, int N>
__device__ __forceinline__ int mx_reaches(const u32x4 (&x)[N][F / 4], unsigned w) {
  unsigned low = 0, high = 0;
  static_for<N>([&](auto f_c) SPT_INLINE {
    constexpr int f = decltype(f_c)::value;
    const int u = mx_reach((w >> (8 * f)) & 255u);
    low |= u == 1 ? mx_numbers<F, N>(x, f) : 0u;
    high |= u == 2 ? mx_numbers<F, N>(x, f) : 0u;
  });
  return 1 | (__any(low != 0) ? 2 : 0) | (__any(high != 0) ? 4 : 0);
}

// mx_bf16 of a block of reach `u`, moved by 2^64 into bf16's range; zeros of another reach.
template <int F, int P>
__device__ __forceinline__ u32x4 mx_bf16_of(u32x4 lo, u32x4 hi, unsigned byte, int u) {
  const bool own = mx_reach(byte) == u;
  const u32x4 r = mx_bf16<F, P>(lo, hi, own ? byte + (unsigned)(u == 1 ? 64 : u == 2 ? -64 : 0) : 127u);
  return own ? r : u32x4{0, 0, 0, 0};
}

// acc += the products of a k-step with far blocks in it: those of each pair of reaches that is there by themselves, and back by their
// power of two. A result without far blocks gets the same bits as without this.
template <int FA, int FB, int FM, int FN>
__device__ __forceinline__ void mx_far_products(const u32x4 (&x)[FM][FA / 4], const u32x4 (&y)[FN][FB / 4], unsigned wa, unsigned wb, f32x4 (&acc)[FM][FN]) {
  const int ra = mx_reaches<FA, FM>(x, wa), rb = mx_reaches<FB, FN>(y, wb);
#pragma unroll 1
  for (int pair = 0; pair < 9; ++pair) {
    const int u = pair / 3, v = pair - 3 * u;
    if (!(ra >> u & 1) || !(rb >> v & 1) || (u == 1 && v == 1)) continue;  // two low ones are below 2^-217: nothing in fp32
    const int back = (u == 1 ? -64 : u == 2 ? 64 : 0) + (v == 1 ? -64 : v == 2 ? 64 : 0);
    static_for<FM>([&](auto i_c) SPT_INLINE {
      constexpr int i = decltype(i_c)::value;
      // what derives from the scales is not kept from pair to pair: it has no registers
      const unsigned sa = opaque_u32(wa), sb = opaque_u32(wb);
      f32x4 d[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j) d[j] = back == 0 ? acc[i][j] : f32x4{0.f, 0.f, 0.f, 0.f};
      static_for<4>([&](auto p_c) SPT_INLINE {
        constexpr int p = decltype(p_c)::value;
        const u32x4 xb = mx_bf16_of<FA, p>(x[i][0], x[i][FA / 4 - 1], (sa >> (8 * i)) & 255u, u);
        static_for<FN>([&](auto j_c) SPT_INLINE {
          constexpr int j = decltype(j_c)::value;
          d[j] = mfma16<__bf16>(xb, mx_bf16_of<FB, p>(y[j][0], y[j][FB / 4 - 1], (sb >> (8 * j)) & 255u, v), d[j]);
        });
      });
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = back == 0 ? d[j][e] : acc[i][j][e] + __builtin_ldexpf(d[j][e], back);
      __builtin_amdgcn_sched_barrier(0);
    });
  }
}

}  // namespace spt
