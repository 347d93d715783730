// Microscaled tensors: quantisation, the values back, and the layout of a checkpoint's codes and scales.
//
// All three are streams: 2 (4) bytes read and 0.53 or 1.03 written per value, or the reverse. A unit is 16 rows by 512
// columns of one workgroup: a wave takes rows w, w + 4, .., a lane eight neighbouring values (16 bytes of fp16 or bf16),
// four lanes a block of 32, so a row's piece is one 1 KiB load and its largest magnitudes two DPP steps. The scales of
// 16 rows of a block lie together in memory and are collected in LDS, so that they leave 16 bytes at a time: written
// row by row each would be a byte in a line of its own.
//   Operands from memory, at the rate of a large copy in brackets: 8192 x 8192 bf16 to 4 bits 29 us (33; the result stays in the last
// cache), to 8 bits 35 (40), 28672 x 8192 to 8 bits 121 (138), 301 x 8190 fp32 to 8 bits 5.4 (2.4); the values of 8192 x 8192 in bf16 from 4
// bits 38 (33), of 28672 x 8192 from 8 bits 123 (138). Units of 64 rows, whose scales leave in whole lines, took, the same operands
// again and again, 34.8 for 28.9, 143 for 119 and 9.6 for 5.0; for values 31.1 and 32.5, but 118 and 115 at 28672 rows and 9.8 and
// 5.1 at 1024 x 4096.
#include "spt_mx_device.h"

namespace spt {

constexpr int kUnitCols = 512;  // 16 blocks
constexpr int kScaleBytes = 16 * kMxUnitRows;  // of a unit

// Word t of a unit's scales, 16 blocks of 16 rows: its place in the tensor, and whether the row has the block.
__device__ __forceinline__ int64_t scale_word(int64_t row0, int cg, int blocks, int t) {
  return (row0 / kMxScaleRows * blocks + cg * 16 + t / 4) * (kMxScaleRows / 4) + row0 % kMxScaleRows / 4 + t % 4;
}
__device__ __forceinline__ bool has_scale_word(int cg, int blocks, int t) { return t < kScaleBytes / 4 && t < (blocks - cg * 16) * 4; }
__device__ __forceinline__ void put_scales(const unsigned* sc, unsigned char* scales, int64_t row0, int cg, int blocks) {
  if (has_scale_word(cg, blocks, threadIdx.x)) ((unsigned*)scales)[scale_word(row0, cg, blocks, threadIdx.x)] = sc[threadIdx.x];
}

template <int T, int BITS>
__global__ void __launch_bounds__(256) mx_quantize_kernel(MxQuantArgs a) {
  __shared__ __attribute__((aligned(16))) unsigned char sc[kScaleBytes];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int groups = (a.blocks + 15) / 16;
  const int64_t row_bytes = (int64_t)a.blocks * (4 * BITS);
  for (int64_t u = blockIdx.x; u < a.units; u += gridDim.x) {
    const int64_t rb = u / groups;
    const int cg = (int)(u - rb * groups);
    const int64_t row0 = rb * kMxUnitRows;
    const int rows = a.rows - row0 >= kMxUnitRows ? kMxUnitRows : a.rows > row0 ? (int)(a.rows - row0) : 0;
    const int col = cg * kUnitCols + lane * 8;
    const bool held = col < a.blocks * kMxBlock;  // the row's padding is written too
    if (rows < kMxUnitRows) {                      // rows behind the last: zeros
      if (threadIdx.x < kScaleBytes / 4) ((unsigned*)sc)[threadIdx.x] = 0;
      __syncthreads();
    }
    float v[4][8];  // the wave's four rows
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = wave + 4 * j;
      load8<T>(a.x + ((row0 + i) * a.ldx + col) * kTypeSize[T], i < rows ? a.k - col : 0, v[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = wave + 4 * j;
      if (i >= rows) break;
      const unsigned s = mx_scale_of<BITS>(v[j]);
      const u32x2 q = mx_codes<BITS>(v[j], s);
      if (held) {
        unsigned char* p = a.codes + (row0 + i) * row_bytes + (int64_t)col * BITS / 8;
        if constexpr (BITS == 8) *(u32x2*)p = q;
        else *(unsigned*)p = q[0];
      }
      if ((lane & 3) == 0) sc[(lane >> 2) * kMxUnitRows + i] = (unsigned char)s;
    }
    __syncthreads();
    put_scales((const unsigned*)sc, a.scales, row0, cg, a.blocks);
    __syncthreads();
  }
}

template <int T, int BITS>
__global__ void __launch_bounds__(256) mx_values_kernel(MxValuesArgs a) {
  __shared__ __attribute__((aligned(16))) unsigned char sc[kScaleBytes];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int groups = (a.blocks + 15) / 16;
  const int64_t row_bytes = (int64_t)a.blocks * (4 * BITS);
  for (int64_t u = blockIdx.x; u < a.units; u += gridDim.x) {
    const int64_t rb = u / groups;
    const int cg = (int)(u - rb * groups);
    const int64_t row0 = rb * kMxUnitRows;
    const int rows = a.rows - row0 >= kMxUnitRows ? kMxUnitRows : a.rows > row0 ? (int)(a.rows - row0) : 0;
    if (has_scale_word(cg, a.blocks, threadIdx.x)) ((unsigned*)sc)[threadIdx.x] = ((const unsigned*)a.scales)[scale_word(row0, cg, a.blocks, threadIdx.x)];
    __syncthreads();
    if constexpr (T == 2) {
      // fp32 leaves in two pieces of 1 KiB a row, four neighbouring values a lane in each (8192 x 8192 from 4 bits, the same codes again:
      // 72 us, 85 with eight neighbours a lane, whose 16-byte stores leave gaps; from memory 80)
      const int col = cg * kUnitCols + lane * 4;
#pragma unroll 4
      for (int i = wave; i < rows; i += 4) {
        const unsigned char* p = a.codes + (row0 + i) * row_bytes + (int64_t)col * BITS / 8;
        u32x2 q = {0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (col + 256 * h < a.k) {
            if constexpr (BITS == 8) q[h] = *(const unsigned*)(p + 256 * h);
            else q[0] |= (unsigned)*(const unsigned short*)(p + 128 * h) << (16 * h);
          }
        float v[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h) mx_values<BITS>(q, sc[(8 * h + (lane >> 3)) * kMxUnitRows + i], v[h]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int left = a.k - (col + 256 * h);
          float* o = (float*)a.out + (row0 + i) * a.ldo + col + 256 * h;
          if (left >= 4) *(u32x4_any*)o = __builtin_bit_cast(u32x4, f32x4{v[h][4 * h], v[h][4 * h + 1], v[h][4 * h + 2], v[h][4 * h + 3]});
          else
            for (int e = 0; e < left; ++e) o[e] = e == 0 ? v[h][4 * h] : e == 1 ? v[h][4 * h + 1] : v[h][4 * h + 2];
        }
      }
      __syncthreads();
      continue;
    }
    const int col = cg * kUnitCols + lane * 8;
    if (col < a.k) {
#pragma unroll 4
      for (int i = wave; i < rows; i += 4) {
        const unsigned char* p = a.codes + (row0 + i) * row_bytes + (int64_t)col * BITS / 8;
        u32x2 q = {0, 0};
        if constexpr (BITS == 8) q = *(const u32x2*)p;
        else q[0] = *(const unsigned*)p;
        float v[8];
        mx_values<BITS>(q, sc[(lane >> 2) * kMxUnitRows + i], v);
        put8<T>(a.out + ((row0 + i) * a.ldo + col) * kTypeSize[T], a.k - col, v);
      }
    }
    __syncthreads();
  }
}

typedef unsigned u32_byte __attribute__((aligned(1)));  // the memory path takes dwords at any byte
typedef unsigned u32x2_byte __attribute__((ext_vector_type(2), aligned(1)));

// Once per weight: a checkpoint's rows may begin anywhere. 28672 x 8192 in 4 bits, from memory: 45 us (48 at the rate of a large copy), in
// 8 bits 85 (94); with each row's last 512 columns taken byte by byte, though all there, 134 and 203.
template <int BITS>
__global__ void __launch_bounds__(256) mx_pack_kernel(MxPackArgs a) {
  __shared__ __attribute__((aligned(16))) unsigned char sc[kScaleBytes];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int groups = (a.blocks + 15) / 16;
  const int row_bytes = a.blocks * 4 * BITS;
  const int64_t used = ((int64_t)a.k * BITS + 7) / 8;  // bytes of a row that hold values
  const int plain = (a.k + kMxBlock - 1) / kMxBlock;
  for (int64_t u = blockIdx.x; u < a.units; u += gridDim.x) {
    const int64_t rb = u / groups;
    const int cg = (int)(u - rb * groups);
    const int64_t row0 = rb * kMxUnitRows;
    const int rows = a.rows - row0 >= kMxUnitRows ? kMxUnitRows : a.rows > row0 ? (int)(a.rows - row0) : 0;
    const int at = (cg * kUnitCols + lane * 8) * BITS / 8;  // the lane's 4 or 8 bytes
    const int si = threadIdx.x >> 4, sb = cg * 16 + (threadIdx.x & 15);  // and a scale of each thread's
    const unsigned char* from = a.codes + (row0 + wave) * a.ldc + at;
    unsigned char* to = a.out_codes + (row0 + wave) * row_bytes + at;
    if (rows == kMxUnitRows && (cg + 1) * kUnitCols <= a.k) {  // all there: the loads before the first is used
      const unsigned char scale = a.scales[(row0 + si) * a.lds + sb];
      unsigned q[4][2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (BITS == 8) {
          const u32x2 v = *(const u32x2_byte*)(from + 4 * j * a.ldc);
          q[j][0] = v[0];
          q[j][1] = v[1];
        } else {
          q[j][0] = *(const u32_byte*)(from + 4 * j * a.ldc);
        }
      }
      sc[(threadIdx.x & 15) * kMxUnitRows + si] = scale;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (BITS == 8) *(u32x2*)(to + 4 * j * row_bytes) = u32x2{q[j][0], q[j][1]};
        else *(unsigned*)(to + 4 * j * row_bytes) = q[j][0];
      }
    } else {
      for (int i = wave; i < rows; i += 4, from += 4 * a.ldc, to += 4 * row_bytes) {
        unsigned q[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < BITS; ++e) {
          unsigned v = at + e < used ? from[e] : 0;
          if (BITS == 4 && at + e == used - 1 && (a.k & 1)) v &= 15;  // an odd row's last byte holds one value
          q[e >> 2] |= v << (8 * (e & 3));
        }
        if (at < row_bytes) {
          ((unsigned*)to)[0] = q[0];
          if (BITS == 8) ((unsigned*)to)[1] = q[1];
        }
      }
      sc[(threadIdx.x & 15) * kMxUnitRows + si] = si < rows && sb < plain ? a.scales[(row0 + si) * a.lds + sb] : 0;
    }
    __syncthreads();
    put_scales((const unsigned*)sc, a.out_scales, row0, cg, a.blocks);
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
const void* mx_pack_fn(int bits) { return bits == 4 ? (const void*)&mx_pack_kernel<4> : (const void*)&mx_pack_kernel<8>; }

}  // namespace spt
