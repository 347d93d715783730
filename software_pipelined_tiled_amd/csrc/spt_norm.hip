// Root-mean-square norm with the residual's addition, its microscaled form, and its gradients.
//
// What bounds them: bytes. A row is read once and stays in registers between the sum of its squares and the result
// (up to 32 values a thread: rows of 32768), so x, the residual, h and y cross memory once each; longer rows are read a
// second time. A workgroup takes neighbouring rows and keeps its columns' weights (and its sums of dweight)
// in registers from row to row. h is rounded to the tensors' type before the statistics: what is normalised is the h that the
// caller gets, as where the addition is an operator of its own. Statistics and products are fp32, y and dx are rounded once.
//
// Gradients: sum h^2 and sum g h come out of one pass, so that r need not be kept by the forward. dweight's sums run
// over a workgroup's rows in registers, leave as one fp32 plane a workgroup, and are added in the planes' order by a second
// kernel: no atomics, the same bits on every run.
#include "spt_mx_device.h"

namespace spt {

// The sum of N values over a workgroup, to all its threads, in a fixed order. `red` holds two sets of N x 16 floats used in
// turn (`turn`), so that one barrier a call is enough.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* red, int turn) {
  float* r = red + turn * N * 16;
  const int waves = blockDim.x >> 6;
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v[i] += __shfl_xor(v[i], d);
  }
  if (waves == 1) return;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i * 16 + (threadIdx.x >> 6)] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float t = 0.f;
    for (int w = 0; w < waves; ++w) t += r[i * 16 + w];
    v[i] = t;
  }
}

// C: pieces of eight values a thread holds of a row (0: rows of any length, in two passes). OUT: 0 y in type T, 4 or 8: MX.
template <int T, int OUT, int C>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(NormArgs a) {
  __shared__ float red[2 * 16];
  constexpr int ES = kTypeSize[T], KEEP = C ? C : 1;
  const int nt = blockDim.x, n = a.n;
  const int pieces = OUT ? a.blocks * (kMxBlock / 8) : (n + 7) / 8;  // an MX row's padding is written too
  const int64_t first = (int64_t)blockIdx.x * a.per, last = first + a.per < a.rows ? first + a.per : a.rows;
  const float inv_n = 1.f / (float)n;

  float w[KEEP][8];
  auto weight = [&](int col, float (&o)[8]) SPT_INLINE {
    if (a.w) {
      load8_any(a.w, a.wtype, col, n - col, o);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = 1.f;
    }
  };
  // h's eight values at `col`, written where a residual is added
  auto h_at = [&](int64_t row, int col, float (&o)[8]) SPT_INLINE {
    load8<T>(a.x + (row * a.ldx + col) * ES, n - col, o);
    if (a.r) {
      float r[8];
      load8<T>(a.r + (row * a.ldr + col) * ES, n - col, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = round_to<T>(o[e] + r[e]);
      put8<T>(a.h + (row * a.ldh + col) * ES, n - col, o);
    }
  };
  auto result = [&](int64_t row, int piece, const float (&h)[8], const float (&wt)[8], float rstd) SPT_INLINE {
    const int col = piece * 8;
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = h[e] * rstd * wt[e];
    if constexpr (OUT == 0) {
      put8<T>(a.y + (row * a.ldy + col) * ES, n - col, y);
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
      if ((threadIdx.x & 3) == 0) {
        unsigned char* sp = a.scales + mx_scale_at(row, piece >> 2, a.blocks);
        *sp = (unsigned char)s;
        if (row == a.rows - 1)  // the rows that fill the last 64: zeros
          for (int64_t i = row % kMxScaleRows + 1; i < kMxScaleRows; ++i) *++sp = 0;
      }
    }
  };

  if constexpr (C > 0) {
#pragma unroll
    for (int c = 0; c < C; ++c) weight((c * nt + (int)threadIdx.x) * 8, w[c]);
  }
  int turn = 0;
  for (int64_t row = first; row < last; ++row, turn ^= 1) {
    float h[KEEP][8], sum[1] = {0.f};
    if constexpr (C > 0) {
#pragma unroll
      for (int c = 0; c < C; ++c) h_at(row, (c * nt + (int)threadIdx.x) * 8, h[c]);
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[0] = __builtin_fmaf(h[c][e], h[c][e], sum[0]);
    } else {
      for (int p = threadIdx.x; p * 8 < n; p += nt) {
        h_at(row, p * 8, h[0]);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[0] = __builtin_fmaf(h[0][e], h[0][e], sum[0]);
      }
    }
    block_sum<1>(sum, red, turn);
    const float rstd = 1.f / __builtin_sqrtf(sum[0] * inv_n + a.eps);
    if constexpr (C > 0) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int p = c * nt + (int)threadIdx.x;
        if (p < pieces) result(row, p, h[c], w[c], rstd);
      }
    } else {
      // what this thread wrote to h, or read from x, a pass before
      const char* src = a.r ? a.h : a.x;
      const int64_t ld = a.r ? a.ldh : a.ldx;
      for (int p = threadIdx.x; p < pieces; p += nt) {
        load8<T>(src + (row * ld + p * 8) * ES, n - p * 8, h[0]);
        weight(p * 8, w[0]);
        result(row, p, h[0], w[0], rstd);
      }
    }
  }
}

template <int T, int C>
__global__ void __launch_bounds__(kNormThreads) norm_grad_kernel(NormGradArgs a) {
  __shared__ float red[2 * 2 * 16];
  constexpr int ES = kTypeSize[T], KEEP = C ? C : 1;
  const int nt = blockDim.x, n = a.n;
  const int64_t first = (int64_t)blockIdx.x * a.per, last = first + a.per < a.rows ? first + a.per : a.rows;
  const float inv_n = 1.f / (float)n;
  float* plane = a.parts ? a.parts + (int64_t)blockIdx.x * n : nullptr;

  auto weight = [&](int col, float (&o)[8]) SPT_INLINE {
    if (a.w) {
      load8_any(a.w, a.wtype, col, n - col, o);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = 1.f;
    }
  };
  float w[KEEP][8], dw[KEEP][8];
  if constexpr (C > 0) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      weight((c * nt + (int)threadIdx.x) * 8, w[c]);
#pragma unroll
      for (int e = 0; e < 8; ++e) dw[c][e] = 0.f;
    }
  }
  // dx's eight values at `col`; t = h r^3 mean(g h) / .. as one factor
  auto grad = [&](int64_t row, int col, const float (&dy)[8], const float (&h)[8], const float (&wt)[8], float rstd, float f) SPT_INLINE {
    float d[8];
    if (a.dh) {
      load8<T>(a.dh + (row * a.lddh + col) * ES, n - col, d);
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] += rstd * (dy[e] * wt[e] - h[e] * f);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] = rstd * (dy[e] * wt[e] - h[e] * f);
    }
    put8<T>(a.dx + (row * a.lddx + col) * ES, n - col, d);
  };
  int turn = 0;
  for (int64_t row = first; row < last; ++row, turn ^= 1) {
    float dy[KEEP][8], h[KEEP][8], sum[2] = {0.f, 0.f};
    auto add = [&](const float (&u)[8], const float (&v)[8], const float (&wt)[8]) SPT_INLINE {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum[0] = __builtin_fmaf(v[e], v[e], sum[0]);
        sum[1] = __builtin_fmaf(u[e] * wt[e], v[e], sum[1]);
      }
    };
    if constexpr (C > 0) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int col = (c * nt + (int)threadIdx.x) * 8;
        load8<T>(a.dy + (row * a.lddy + col) * ES, n - col, dy[c]);
        load8<T>(a.h + (row * a.ldh + col) * ES, n - col, h[c]);
      }
#pragma unroll
      for (int c = 0; c < C; ++c) add(dy[c], h[c], w[c]);
    } else {
      for (int p = threadIdx.x; p * 8 < n; p += nt) {
        load8<T>(a.dy + (row * a.lddy + p * 8) * ES, n - p * 8, dy[0]);
        load8<T>(a.h + (row * a.ldh + p * 8) * ES, n - p * 8, h[0]);
        weight(p * 8, w[0]);
        add(dy[0], h[0], w[0]);
      }
    }
    block_sum<2>(sum, red, turn);
    const float rstd = 1.f / __builtin_sqrtf(sum[0] * inv_n + a.eps);
    const float f = rstd * rstd * (sum[1] * inv_n);
    if constexpr (C > 0) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int col = (c * nt + (int)threadIdx.x) * 8;
        if (a.dx && col < n) grad(row, col, dy[c], h[c], w[c], rstd, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[c][e] = __builtin_fmaf(dy[c][e], h[c][e] * rstd, dw[c][e]);
      }
    } else {
      for (int p = threadIdx.x; p * 8 < n; p += nt) {
        const int col = p * 8;
        load8<T>(a.dy + (row * a.lddy + col) * ES, n - col, dy[0]);
        load8<T>(a.h + (row * a.ldh + col) * ES, n - col, h[0]);
        weight(col, w[0]);
        if (a.dx) grad(row, col, dy[0], h[0], w[0], rstd, f);
        if (plane) {  // the plane's columns are this thread's alone
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (col + e < n) plane[col + e] = __builtin_fmaf(dy[0][e], h[0][e] * rstd, row == first ? 0.f : plane[col + e]);
        }
      }
    }
  }
  if constexpr (C > 0) {
    if (plane) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int col = (c * nt + (int)threadIdx.x) * 8;
        put8<2>((char*)(plane + col), n - col, dw[c]);
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
  const bool vec = a.n % 4 == 0 && col + 4 <= a.n;
  for (int p = p0; p < a.count; p += 64) {
    const float* src = a.parts + (int64_t)p * a.n + col;
    if (vec) {
      const f32x4 v = *(const f32x4*)src;
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] += v[e];
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
  return c == 1 ? (const void*)&norm_kernel<T, OUT, 1> : c == 2 ? (const void*)&norm_kernel<T, OUT, 2>
       : c == 4 ? (const void*)&norm_kernel<T, OUT, 4> : c == 8 ? (const void*)&norm_kernel<T, OUT, 8> : (const void*)&norm_kernel<T, OUT, 0>;
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
  return c == 1 ? (const void*)&norm_grad_kernel<T, 1> : c == 2 ? (const void*)&norm_grad_kernel<T, 2>
       : c == 4 ? (const void*)&norm_grad_kernel<T, 4> : (const void*)&norm_grad_kernel<T, 0>;
}
const void* norm_grad_fn(int dtype, int c) {
  return dtype == 0 ? norm_grad_pick<0>(c) : dtype == 1 ? norm_grad_pick<1>(c) : norm_grad_pick<2>(c);
}
const void* norm_parts_fn() { return (const void*)&norm_parts_kernel; }

}  // namespace spt
