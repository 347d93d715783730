// Microscaled tensors: quantisation, the values back, and the layout of a checkpoint's codes and scales.
//
// All three are streams: 2 (4) bytes read and 0.53 or 1.03 written per value, or the reverse. A unit is 64 rows by 512
// columns of one workgroup: a wave takes rows w, w + 4, .., a lane eight neighbouring values (16 bytes of fp16 or bf16),
// four lanes a block of 32, so a row's piece is one 1 KiB load and its largest magnitudes two DPP steps. The scales of
// 64 rows by 16 blocks lie together in memory and are collected in LDS, so that they leave in one piece of 1 KiB: written
// row by row each would be a byte in a line of its own.
#include "spt_mx_device.h"

namespace spt {

constexpr int kUnitCols = 512;  // 16 blocks

// Copies the unit's 16 x 64 scale bytes out of LDS.
__device__ __forceinline__ void put_scales(const unsigned* sc, unsigned char* scales, int64_t rb, int cg, int blocks) {
  const int first = cg * 16, count = blocks - first < 16 ? blocks - first : 16;
  unsigned* dst = (unsigned*)(scales + (rb * blocks + first) * kMxScaleRows);
  if ((int)threadIdx.x < count * 16) dst[threadIdx.x] = sc[threadIdx.x];
}

template <int T, int BITS>
__global__ void __launch_bounds__(256) mx_quantize_kernel(MxQuantArgs a) {
  __shared__ __attribute__((aligned(16))) unsigned char sc[16 * kMxScaleRows];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int groups = (a.blocks + 15) / 16;
  const int64_t row_bytes = (int64_t)a.blocks * (4 * BITS);
  for (int64_t u = blockIdx.x; u < a.units; u += gridDim.x) {
    const int64_t rb = u / groups;
    const int cg = (int)(u - rb * groups);
    const int64_t row0 = rb * kMxScaleRows;
    const int rows = a.rows - row0 < kMxScaleRows ? (int)(a.rows - row0) : kMxScaleRows;
    const int col = cg * kUnitCols + lane * 8;
    const bool held = col < a.blocks * kMxBlock;  // the row's padding is written too
    if (rows < kMxScaleRows) {                     // rows behind the last: zeros
      ((unsigned*)sc)[threadIdx.x] = 0;
      __syncthreads();
    }
    for (int base = wave; base < rows; base += 16) {  // four rows' loads before the first is used
      float v[4][8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = base + 4 * j;
        load8<T>(a.x + ((row0 + i) * a.ldx + col) * kTypeSize[T], i < rows ? a.k - col : 0, v[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = base + 4 * j;
        if (i >= rows) break;
        const unsigned s = mx_scale_of<BITS>(v[j]);
        const u32x2 q = mx_codes<BITS>(v[j], s);
        if (held) {
          unsigned char* p = a.codes + (row0 + i) * row_bytes + (int64_t)col * BITS / 8;
          if constexpr (BITS == 8) *(u32x2*)p = q;
          else *(unsigned*)p = q[0];
        }
        if ((lane & 3) == 0) sc[(lane >> 2) * kMxScaleRows + i] = (unsigned char)s;
      }
    }
    __syncthreads();
    put_scales((const unsigned*)sc, a.scales, rb, cg, a.blocks);
    __syncthreads();
  }
}

template <int T, int BITS>
__global__ void __launch_bounds__(256) mx_values_kernel(MxValuesArgs a) {
  __shared__ __attribute__((aligned(16))) unsigned char sc[16 * kMxScaleRows];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int groups = (a.blocks + 15) / 16;
  const int64_t row_bytes = (int64_t)a.blocks * (4 * BITS);
  for (int64_t u = blockIdx.x; u < a.units; u += gridDim.x) {
    const int64_t rb = u / groups;
    const int cg = (int)(u - rb * groups);
    const int64_t row0 = rb * kMxScaleRows;
    const int rows = a.rows - row0 < kMxScaleRows ? (int)(a.rows - row0) : kMxScaleRows;
    const int first = cg * 16, count = a.blocks - first < 16 ? a.blocks - first : 16;
    const unsigned* src = (const unsigned*)(a.scales + (rb * a.blocks + first) * kMxScaleRows);
    if ((int)threadIdx.x < count * 16) ((unsigned*)sc)[threadIdx.x] = src[threadIdx.x];
    __syncthreads();
    const int col = cg * kUnitCols + lane * 8;
    if (col < a.k) {
#pragma unroll 4
      for (int i = wave; i < rows; i += 4) {
        const unsigned char* p = a.codes + (row0 + i) * row_bytes + (int64_t)col * BITS / 8;
        u32x2 q = {0, 0};
        if constexpr (BITS == 8) q = *(const u32x2*)p;
        else q[0] = *(const unsigned*)p;
        float v[8];
        mx_values<BITS>(q, sc[(lane >> 2) * kMxScaleRows + i], v);
        put8<T>(a.out + ((row0 + i) * a.ldo + col) * kTypeSize[T], a.k - col, v);
      }
    }
    __syncthreads();
  }
}

// Once per weight: byte loads, so that a checkpoint's rows may begin anywhere.
__global__ void __launch_bounds__(256) mx_pack_kernel(MxPackArgs a) {
  __shared__ __attribute__((aligned(16))) unsigned char sc[16 * kMxScaleRows];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int groups = (a.blocks + 15) / 16;
  const int row_bytes = a.blocks * 4 * a.bits;
  const int64_t used = ((int64_t)a.k * a.bits + 7) / 8;  // bytes of a row that hold values
  const int plain = (a.k + kMxBlock - 1) / kMxBlock;
  for (int64_t u = blockIdx.x; u < a.units; u += gridDim.x) {
    const int64_t rb = u / groups;
    const int cg = (int)(u - rb * groups);
    const int64_t row0 = rb * kMxScaleRows;
    const int rows = a.rows - row0 < kMxScaleRows ? (int)(a.rows - row0) : kMxScaleRows;
    const int at = (cg * kUnitCols + lane * 8) * a.bits / 8;  // the lane's 4 or 8 bytes
    for (int i = wave; i < rows; i += 4) {
      const unsigned char* p = a.codes + (row0 + i) * a.ldc;
      unsigned q[2] = {0, 0};
      for (int e = 0; e < a.bits; ++e) {
        const int64_t b = at + e;
        unsigned v = b < used ? p[b] : 0;
        if (a.bits == 4 && b == used - 1 && (a.k & 1)) v &= 15;  // an odd row's last byte holds one value
        q[e >> 2] |= v << (8 * (e & 3));
      }
      if (at < row_bytes) {
        unsigned* o = (unsigned*)(a.out_codes + (row0 + i) * row_bytes + at);
        o[0] = q[0];
        if (a.bits == 8) o[1] = q[1];
      }
    }
    for (int t = threadIdx.x; t < 16 * kMxScaleRows; t += 256) {
      const int i = t >> 4, b = cg * 16 + (t & 15);
      sc[(t & 15) * kMxScaleRows + i] = i < rows && b < plain ? a.scales[(row0 + i) * a.lds + b] : 0;
    }
    __syncthreads();
    put_scales((const unsigned*)sc, a.out_scales, rb, cg, a.blocks);
    __syncthreads();
  }
}

const void* mx_quantize_fn(int dtype, int bits) {
  if (bits == 4) return dtype == 0 ? (const void*)&mx_quantize_kernel<0, 4> : dtype == 1 ? (const void*)&mx_quantize_kernel<1, 4> : (const void*)&mx_quantize_kernel<2, 4>;
  return dtype == 0 ? (const void*)&mx_quantize_kernel<0, 8> : dtype == 1 ? (const void*)&mx_quantize_kernel<1, 8> : (const void*)&mx_quantize_kernel<2, 8>;
}
const void* mx_values_fn(int dtype, int bits) {
  if (bits == 4) return dtype == 0 ? (const void*)&mx_values_kernel<0, 4> : dtype == 1 ? (const void*)&mx_values_kernel<1, 4> : (const void*)&mx_values_kernel<2, 4>;
  return dtype == 0 ? (const void*)&mx_values_kernel<0, 8> : dtype == 1 ? (const void*)&mx_values_kernel<1, 8> : (const void*)&mx_values_kernel<2, 8>;
}
const void* mx_pack_fn() { return (const void*)&mx_pack_kernel; }

}  // namespace spt
