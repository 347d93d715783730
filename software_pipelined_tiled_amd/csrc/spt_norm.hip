// Root-mean-square norm with the residual's addition, its microscaled form, and its gradients.
//
// What bounds them: bytes. A row is read once and stays in registers, as it lies in memory, between the sum of its squares and
// the result, so x, the residual, h and y cross memory once each; rows of more than 32768 16-bit or 16384 fp32 values
// are read a second time. h is rounded to the tensors' type before the statistics: what is normalised is the h that the
// caller gets, as where the addition is an operator of its own. Statistics and products are fp32, y and dx are rounded once.
//
// A workgroup has a row at a time, and takes several neighbouring rows, the next one's loads in flight while it adds up the
// squares; rows of up to 512 values are a wave's or a part of one, several to a workgroup (30000 rows of 200 from the last cache: 9.8
// us, 26 with a wave to a row). Weights stay in registers from row to row where rows are short enough, and else come from the L2. With the
// residual, operands from memory, at the rate of a large copy (5.16 TB/s) in brackets: 8191 rows of 8192 fp16 106 us (104), as MX of 8
// bits 97 (92), of 4 bits 92 (85); 8192 rows of 4096 bf16 56, 47 and 46 (52, 46, 43); 2000 rows of 28672 bf16 99 (89; 4 us more without the
// loads ahead), as MX of 8 bits 103 (78: its four pieces have no loads ahead, and the row ends' lane masks, kept over the rows, fill the
// scalar registers: 128 are spilled); 1003 rows of 4097 fp32 17 (13); 1000 rows of 38400 fp16 in two passes 80 (60).
//
// Gradients: sum h^2 and sum g h come out of one pass, so that r need not be kept by the forward. dweight's sums run
// over a workgroup's rows in registers, for rows of more than 16384 values in LDS, and in its plane in memory for those that the
// LDS does not hold either; they leave as one fp32 plane a workgroup, and are added in the planes' order by a second
// kernel: no atomics, the same bits on every run. A workgroup has eight rows or more, so that the planes are few, with few rows side
// by side. With dh, from memory: 8191 rows of 8192 fp16 113 us (104), 8192 of 4096 bf16 59 (52), 2000 of 28672 bf16 138 (89: each row's dy
// and h are read twice, with nothing in flight from one row to the next; 185 with the sums in registers, which did not fit), 300 rows
// of 4096 10.5 (1.9: two launches).
#include "spt_mx_device.h"

namespace spt {

constexpr int kShort = -1;  // C of rows that a part of a wave holds
constexpr int kLds = -2;    // gradients: C of long rows with dweight's sums in LDS
constexpr int kSide = -3;   // gradients: C of rows of several waves, with several of them side by side in a workgroup

template <int CTRL>
__device__ __forceinline__ float lanes_moved(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

// The sum of N values over the `lanes` threads of a row (a power of two up to 64, or all the workgroup's), to all of them, in a fixed
// order: in pairs, of the waves' sums too (one after the other they are off by 1.5 times as much in the mean). `red` holds two sets of
// N x 16 floats used in turn (`turn`), so that one barrier a call is enough. `wave0`: the row's first wave.
template <int N, bool SHORT>
__device__ __forceinline__ void row_sum(float (&v)[N], float* red, int turn, int lanes, int wave0 = 0) {
  if constexpr (SHORT) {
    for (int d = lanes >> 1; d >= 1; d >>= 1) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], d);
    }
  } else {
    float* r = red + turn * N * 16;
    const int waves = lanes >> 6;
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) v[i] += __shfl_xor(v[i], d);
    }
    if (blockDim.x == 64) return;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) r[i * 16 + (threadIdx.x >> 6)] = v[i];
    }
    __syncthreads();
    const int w = threadIdx.x & 15;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float t = w < waves ? r[i * 16 + wave0 + w] : 0.f;
      t += lanes_moved<0xB1>(t);         // lanes 1 0 3 2 of four
      t += lanes_moved<0x4E>(t);         // lanes 2 3 0 1
      t += lanes_moved<0x141>(t);        // eight lanes backwards: the other four's sum
      v[i] = t + lanes_moved<0x140>(t);  // sixteen lanes backwards: the other eight's
    }
  }
}

__device__ __forceinline__ void load_weight(const char* w, int type, int col, int n, float (&o)[8]) {
  if (w) {
    load8_any(w, type, col, n - col, o);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = 1.f;
  }
}

// C: pieces of eight values a thread holds of a row (kShort: one, rows of part of a wave; 0: rows of any length, in two passes).
// OUT: 0 y in type T, 4 or 8: MX.
template <int T, int OUT, int C>
__global__ void __launch_bounds__(C == 0 ? 512 : 1024) norm_kernel(NormArgs a) {
  __shared__ float red[2 * 16];
  constexpr bool SHORT = C == kShort;
  constexpr int ES = kTypeSize[T], P = SHORT ? 1 : C, KEEP = P ? P : 1;
  constexpr bool W_KEPT = P == 1 || P == 2;
  const int n = a.n, lanes = SHORT ? a.lanes : blockDim.x, at = threadIdx.x & (SHORT ? lanes - 1 : 1023);
  const int pieces = OUT ? a.blocks * (kMxBlock / 8) : (n + 7) / 8;  // an MX row's padding is written too
  // this thread's first row, the last row of its workgroup, and from row to row
  const int step = SHORT ? blockDim.x / lanes : 1;
  const int64_t first = (int64_t)blockIdx.x * a.per + (SHORT ? threadIdx.x / lanes : 0);
  const int64_t last = ((int64_t)blockIdx.x + 1) * a.per < a.rows ? ((int64_t)blockIdx.x + 1) * a.per : a.rows;
  const float inv_n = 1.f / (float)n;

  auto col_of = [&](int c) SPT_INLINE { return (c * lanes + at) * 8; };
  float w[W_KEPT ? KEEP : 1][8];
  if constexpr (W_KEPT) {
#pragma unroll
    for (int c = 0; c < P; ++c) load_weight(a.w, a.wtype, col_of(c), n, w[c]);
  }
  // h's eight values at `col` from x's and the residual's
  auto sum_of = [&](int64_t row, int col, const Raw8<T>& x, const Raw8<T>& r) SPT_INLINE {
    if (!a.r) return x;
    float u[8], v[8];
    unpack<T>(x, u);
    unpack<T>(r, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] += v[e];
    const Raw8<T> h = pack<T>(u);
    put_raw<T>(a.h + row * a.ldh * ES + (unsigned)(col * ES), n - col, h);
    return h;
  };
  auto square = [&](const Raw8<T>& h, float& s) SPT_INLINE {
    float v[8];
    unpack<T>(h, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = __builtin_fmaf(v[e], v[e], s);
  };
  // scales of a thread's last four rows, the newest on top: they leave as words (8192 rows of 4096 bf16: 44 us, 48 with a byte a row)
  constexpr bool WORDS = OUT != 0 && P > 0 && !SHORT;
  unsigned kept[WORDS ? KEEP : 1];
  auto put_scale = [&](int64_t row, int piece, unsigned s, unsigned& word) SPT_INLINE {
    unsigned char* sp = a.scales + mx_scale_at(row, piece >> 2, a.blocks);
    if constexpr (WORDS) {
      word = word >> 8 | s << 24;
      const int turn = (int)(row & 3), count = row - first < turn ? (int)(row - first) + 1 : turn + 1;  // rows of the word that are here
      if (turn != 3 && row != last - 1) return;
      if (count == 4) *(unsigned*)(sp - 3) = word;
      else if (count == 1) *sp = (unsigned char)s;
      else
        for (int i = 0; i < count; ++i) sp[-i] = (unsigned char)(word >> (24 - 8 * i));
    } else {
      *sp = (unsigned char)s;
    }
    if (row == a.rows - 1)  // the rows that fill the last 64: zeros
      for (int64_t i = row % kMxScaleRows + 1; i < kMxScaleRows; ++i) *++sp = 0;
  };
  auto result = [&](int64_t row, int piece, const Raw8<T>& h, const float (&wt)[8], float rstd, unsigned& word) SPT_INLINE {
    const int col = piece * 8;
    float y[8];
    unpack<T>(h, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = y[e] * rstd * wt[e];
    if constexpr (OUT == 0) {
      put8<T>(a.y + row * a.ldy * ES + (unsigned)(col * ES), n - col, y);
    } else {
      // columns behind n have to be zeros also where the row's factor is not finite
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e >= n - col) y[e] = 0.f;
      const unsigned s = mx_scale_of<OUT>(y);
      const u32x2 q = mx_codes<OUT>(y, s);
      unsigned char* p = (unsigned char*)a.y + row * ((int64_t)a.blocks * (4 * OUT)) + (int64_t)piece * OUT;
      if constexpr (OUT == 8) *(u32x2*)p = q;
      else *(unsigned*)p = q[0];
      if ((threadIdx.x & 3) == 0) put_scale(row, piece, s, word);
    }
  };

  int turn = 0;
  if constexpr (P > 0) {
    constexpr bool AHEAD = P <= 2 || OUT == 0;  // the next row's loads before this row's sum (the MX form of four pieces has no registers for it)
    Raw8<T> x[KEEP], r[KEEP];
    auto fetch = [&](int64_t row) SPT_INLINE {
#pragma unroll
      for (int c = 0; c < P; ++c) {
        const int col = col_of(c);
        x[c] = load_ahead<T>(a.x + row * a.ldx * ES, col, n);
        if (a.r) r[c] = load_ahead<T>(a.r + row * a.ldr * ES, col, n);
      }
    };
    if (AHEAD && first < last) fetch(first);
    for (int64_t row = first; row < last; row += step, turn ^= 1) {
      if (!AHEAD) fetch(row);
      Raw8<T> h[KEEP];
      float sum[1] = {0.f};
#pragma unroll
      for (int c = 0; c < P; ++c) {
        settle<T>(x[c], col_of(c), n);
        if (a.r) settle<T>(r[c], col_of(c), n);
        h[c] = sum_of(row, col_of(c), x[c], r[c]);
        square(h[c], sum[0]);
      }
      if (AHEAD && row + step < last) fetch(row + step);
      row_sum<1, SHORT>(sum, red, turn, lanes);
      const char* wp = a.w;
      if constexpr (!W_KEPT) asm volatile("" : "+s"(wp));  // loaded for each row: out of the loop they would be kept all the same
      const float rstd = 1.f / __builtin_sqrtf(sum[0] * inv_n + a.eps);
#pragma unroll
      for (int c = 0; c < P; ++c) {
        const int piece = c * lanes + at;
        if (piece >= pieces) continue;
        if constexpr (W_KEPT) {
          result(row, piece, h[c], w[c], rstd, kept[WORDS ? c : 0]);
        } else {
          load_weight(wp, a.wtype, piece * 8, n, w[0]);
          result(row, piece, h[c], w[0], rstd, kept[WORDS ? c : 0]);
        }
      }
    }
  } else {
    for (int64_t row = first; row < last; ++row, turn ^= 1) {
      float sum[1] = {0.f};
      for (int p = threadIdx.x; p * 8 < n; p += lanes) {
        const int col = p * 8;
        Raw8<T> x = load_ahead<T>(a.x + row * a.ldx * ES, col, n), r = x;
        if (a.r) {
          r = load_ahead<T>(a.r + row * a.ldr * ES, col, n);
          settle<T>(r, col, n);
        }
        settle<T>(x, col, n);
        square(sum_of(row, col, x, r), sum[0]);
      }
      row_sum<1, false>(sum, red, turn, lanes);
      const float rstd = 1.f / __builtin_sqrtf(sum[0] * inv_n + a.eps);
      // what this thread wrote to h, or read from x, a pass before
      const char* src = a.r ? a.h : a.x;
      const int64_t ld = a.r ? a.ldh : a.ldx;
      for (int p = threadIdx.x; p < pieces; p += lanes) {
        const Raw8<T> h = load_raw<T>(src + row * ld * ES + (unsigned)((p * 8) * ES), n - p * 8);
        load_weight(a.w, a.wtype, p * 8, n, w[0]);
        result(row, p, h, w[0], rstd, kept[0]);
      }
    }
  }
}

// C as above, kLds and kSide.
template <int T, int C>
__global__ void __launch_bounds__(C == 0 ? 512 : 1024) norm_grad_kernel(NormGradArgs a) {
  __shared__ float red[2 * 2 * 16];
  constexpr bool SHORT = C == kShort, SIDE = C == kSide, SEVERAL = SHORT || SIDE;
  constexpr int ES = kTypeSize[T], P = SEVERAL ? 1 : C == kLds ? 0 : C, KEEP = P ? P : 1;
  constexpr bool W_KEPT = P == 1;
  const int n = a.n, lanes = SEVERAL ? a.lanes : blockDim.x;
  const int place = SHORT ? threadIdx.x / lanes : SIDE ? __builtin_amdgcn_readfirstlane(threadIdx.x / lanes) : 0;  // among the rows side by side
  const int at = threadIdx.x - place * lanes;
  const int step = SEVERAL ? blockDim.x / lanes : 1;
  const int64_t first = (int64_t)blockIdx.x * a.per + place;
  const int64_t last = ((int64_t)blockIdx.x + 1) * a.per < a.rows ? ((int64_t)blockIdx.x + 1) * a.per : a.rows;
  const float inv_n = 1.f / (float)n;
  float* plane = a.parts ? a.parts + (int64_t)blockIdx.x * n : nullptr;

  auto col_of = [&](int c) SPT_INLINE { return (c * lanes + at) * 8; };
  float w[1][8];
  if constexpr (W_KEPT) load_weight(a.w, a.wtype, col_of(0), n, w[0]);
  auto add = [&](const Raw8<T>& dy, const Raw8<T>& h, const float (&wt)[8], float (&sum)[2]) SPT_INLINE {
    float u[8], v[8];
    unpack<T>(dy, u);
    unpack<T>(h, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sum[0] = __builtin_fmaf(v[e], v[e], sum[0]);
      sum[1] = __builtin_fmaf(u[e] * wt[e], v[e], sum[1]);
    }
  };
  // dx's eight values at `col`, with f = r^2 mean(g h)
  auto grad = [&](int64_t row, int col, const Raw8<T>& dy, const Raw8<T>& h, const Raw8<T>& dh, const float (&wt)[8], float rstd,
                  float f) SPT_INLINE {
    float u[8], v[8], d[8];
    unpack<T>(dy, u);
    unpack<T>(h, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = rstd * (u[e] * wt[e] - v[e] * f);
    if (a.dh) {
      unpack<T>(dh, d);
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] += d[e];
    }
    put8<T>(a.dx + row * a.lddx * ES + (unsigned)(col * ES), n - col, u);
  };
  int turn = 0;
  if constexpr (P > 0) {
    float dw[KEEP][8];
#pragma unroll
    for (int c = 0; c < P; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) dw[c][e] = 0.f;
    constexpr bool AHEAD = P == 1;  // the next row's loads before this row's sum
    Raw8<T> dy[KEEP], h[KEEP], dh[KEEP], u, v;
    auto fetch = [&](int64_t row, int c, Raw8<T>& p, Raw8<T>& q) SPT_INLINE {
      const int col = col_of(c);
      p = load_ahead<T>(a.dy + row * a.lddy * ES, col, n);
      q = load_ahead<T>(a.h + row * a.ldh * ES, col, n);
    };
    if (AHEAD && first < last) fetch(first, 0, dy[0], h[0]);
    // rows of several waves side by side meet at barriers: all go on to the workgroup's last row
    for (int64_t row = first; (SIDE ? row - place : row) < last; row += step, turn ^= 1) {
      const bool live = !SIDE || row < last;
      float sum[2] = {0.f, 0.f};
      const char* wp = a.w;
      if constexpr (!W_KEPT) asm volatile("" : "+s"(wp));  // loaded for each row: out of the loop they would be kept all the same
      if constexpr (!AHEAD) {
#pragma unroll
        for (int c = 0; c < P; ++c) fetch(row, c, dy[c], h[c]);
      }
#pragma unroll
      for (int c = 0; c < P; ++c) {
        if (!live) break;
        const int col = col_of(c);
        if (a.dh) dh[c] = load_ahead<T>(a.dh + row * a.lddh * ES, col, n);
        settle<T>(dy[c], col, n);
        settle<T>(h[c], col, n);
        if constexpr (!W_KEPT) load_weight(wp, a.wtype, col, n, w[0]);
        add(dy[c], h[c], w[0], sum);
      }
      if (AHEAD && row + step < last) fetch(row + step, 0, u, v);
      row_sum<2, SHORT>(sum, red, turn, lanes, SIDE ? place * (lanes >> 6) : 0);
      if (!live) continue;
      const float rstd = 1.f / __builtin_sqrtf(sum[0] * inv_n + a.eps);
      const float f = rstd * rstd * (sum[1] * inv_n);
#pragma unroll
      for (int c = 0; c < P; ++c) {
        const int col = col_of(c);
        if constexpr (!W_KEPT) load_weight(wp, a.wtype, col, n, w[0]);
        if (a.dx && col < n) {
          if (a.dh) settle<T>(dh[c], col, n);
          grad(row, col, dy[c], h[c], dh[c], w[0], rstd, f);
        }
        float p[8], q[8];
        unpack<T>(dy[c], p);
        unpack<T>(h[c], q);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[c][e] = __builtin_fmaf(p[e], q[e] * rstd, dw[c][e]);
      }
      if constexpr (AHEAD) dy[0] = u, h[0] = v;
    }
    if constexpr (SEVERAL) {  // the rows' parts of the workgroup, in their order
      __shared__ float part[(SIDE ? 1024 : 256) * 8];
#pragma unroll
      for (int e = 0; e < 8; ++e) part[threadIdx.x * 8 + e] = dw[0][e];
      __syncthreads();
      if (plane && (int)threadIdx.x < lanes) {
        for (int s = 1; s < step; ++s)
#pragma unroll
          for (int e = 0; e < 8; ++e) dw[0][e] += part[(s * lanes + at) * 8 + e];
        put8<2>((char*)(plane + at * 8), n - at * 8, dw[0]);
      }
    } else if (plane) {
#pragma unroll
      for (int c = 0; c < P; ++c) put8<2>((char*)(plane + col_of(c)), n - col_of(c), dw[c]);
    }
  } else {
    extern __shared__ u32x4 sums[];  // kLds: two to a piece, the first ones of all pieces before the second ones
    const int pieces = (n + 7) / 8;
    for (int64_t row = first; row < last; ++row, turn ^= 1) {
      float sum[2] = {0.f, 0.f};
      auto piece = [&](int col, Raw8<T>& u, Raw8<T>& v) SPT_INLINE {
        u = load_ahead<T>(a.dy + row * a.lddy * ES, col, n);
        v = load_ahead<T>(a.h + row * a.ldh * ES, col, n);
        load_weight(a.w, a.wtype, col, n, w[0]);
        settle<T>(u, col, n);
        settle<T>(v, col, n);
      };
      Raw8<T> u, v;
      for (int p = threadIdx.x; p * 8 < n; p += lanes) {
        piece(p * 8, u, v);
        add(u, v, w[0], sum);
      }
      row_sum<2, false>(sum, red, turn, lanes);
      const float rstd = 1.f / __builtin_sqrtf(sum[0] * inv_n + a.eps);
      const float f = rstd * rstd * (sum[1] * inv_n);
      for (int p = threadIdx.x; p * 8 < n; p += lanes) {
        const int col = p * 8;
        piece(col, u, v);
        // dx may be dy's own memory: dweight's part is taken from what was read
        Raw8<T> d = u;
        if (a.dh) {
          d = load_ahead<T>(a.dh + row * a.lddh * ES, col, n);
          settle<T>(d, col, n);
        }
        if (a.dx) grad(row, col, u, v, d, w[0], rstd, f);
        if (plane) {  // a piece's sums are this thread's alone
          float p8[8], q8[8], s8[8];
          unpack<T>(u, p8);
          unpack<T>(v, q8);
          if (row > first) {
            if constexpr (C == kLds) unpack<2>(Raw8<2>{sums[p], sums[pieces + p]}, s8);
            else load8<2>((const char*)(plane + col), n - col, s8);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) s8[e] = __builtin_fmaf(p8[e], q8[e] * rstd, row > first ? s8[e] : 0.f);
          if (C == kLds && row + 1 < last) {
            const Raw8<2> r8 = pack<2>(s8);
            sums[p] = r8.q[0];
            sums[pieces + p] = r8.q[1];
          } else {
            put8<2>((char*)(plane + col), n - col, s8);
          }
        }
      }
    }
  }
}

// dweight = the planes' sum: a workgroup has 16 columns, 4 to a lane group of 64 lanes that share out the planes (64 bytes
// of a plane a row); the lanes' sums are added in their order.
__global__ void __launch_bounds__(256) norm_parts_kernel(NormPartsArgs a) {
  __shared__ float red[64][17];
  const int c = threadIdx.x & 3, p0 = threadIdx.x >> 2;
  const int col = blockIdx.x * 16 + c * 4;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  for (int p = p0; p < a.count; p += 64) {
    const float* src = a.parts + (int64_t)p * a.n + col;
    if (col + 4 <= a.n) {
      const u32x4 v = *(const u32x4_any*)src;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const unsigned word = v[e];
        s[e] += __builtin_bit_cast(float, word);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + e < a.n) s[e] += src[e];
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) red[p0][c * 4 + e] = s[e];
  __syncthreads();
  if (threadIdx.x < 16 && blockIdx.x * 16 + (int)threadIdx.x < a.n) {
    float t = 0.f;
    for (int p = 0; p < 64; ++p) t += red[p][threadIdx.x];
    const int64_t at = (int64_t)blockIdx.x * 16 + threadIdx.x;
    if (a.wtype == 2) ((float*)a.out)[at] = t;
    else ((unsigned short*)a.out)[at] = (unsigned short)((a.wtype == 1 ? pack_bf16(t, 0.f) : pack_f16(t, 0.f)) & 0xFFFFu);
  }
}

template <int T, int OUT>
static const void* norm_pick(int c) {
  if constexpr (T != 2)
    if (c == 4) return (const void*)&norm_kernel<T, OUT, 4>;
  switch (c) {
    case kShort: return (const void*)&norm_kernel<T, OUT, kShort>;
    case 1: return (const void*)&norm_kernel<T, OUT, 1>;
    case 2: return (const void*)&norm_kernel<T, OUT, 2>;
    default: return (const void*)&norm_kernel<T, OUT, 0>;
  }
}
template <int T>
static const void* norm_pick_out(int out, int c) {
  return out == 0 ? norm_pick<T, 0>(c) : out == 4 ? norm_pick<T, 4>(c) : norm_pick<T, 8>(c);
}
const void* norm_fn(int dtype, int out, int c) {
  return dtype == 0 ? norm_pick_out<0>(out, c) : dtype == 1 ? norm_pick_out<1>(out, c) : norm_pick_out<2>(out, c);
}
template <int T>
static const void* norm_grad_pick(int c) {
  switch (c) {
    case kShort: return (const void*)&norm_grad_kernel<T, kShort>;
    case 1: return (const void*)&norm_grad_kernel<T, 1>;
    case 2: return (const void*)&norm_grad_kernel<T, 2>;
    case kLds: return (const void*)&norm_grad_kernel<T, kLds>;
    case kSide: return (const void*)&norm_grad_kernel<T, kSide>;
    default: return (const void*)&norm_grad_kernel<T, 0>;
  }
}
const void* norm_grad_fn(int dtype, int c) {
  return dtype == 0 ? norm_grad_pick<0>(c) : dtype == 1 ? norm_grad_pick<1>(c) : norm_grad_pick<2>(c);
}
const void* norm_parts_fn() { return (const void*)&norm_parts_kernel; }

}  // namespace spt
