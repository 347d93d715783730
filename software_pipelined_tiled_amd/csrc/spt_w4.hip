// Products with 4-bit weights and group scales:
//   y[i][n] = sum over k of x[i][k] * (q[n][k] - z[n][k / G]) * s[n][k / G]
// for one weight matrix, or one per expert over rows sorted by expert. q and z are 0 .. 15 (z = 8
// where there are none), s and x 16-bit, G = 32, 64 or 128.
//
// Arithmetic. q - z is a whole number of at most four bits and a sign: it is exact in fp16 and in
// bf16. So the matrix instruction takes x and q - z, every product is exact, and the sum over one
// group stays in its fp32 accumulator; the group's scale multiplies that sum in fp32. No weight is
// rounded, a column whose weights all equal their zero point gives exact zeros, and infinities and
// NaN in x travel as in the formula (a group's sum of x times q - z has to stay inside fp32's range).
//
// What bounds it: with few rows, reading the weights (half a byte each). The packed layout gives
// each lane 16 consecutive bytes of the stream, which are the weights of four matrix instructions
// (32 k each) in the lane's own operand position, so a wave reads 1 KiB (16 columns x 128 k) per
// load and nothing passes through LDS. Turning four bits into an operand costs 9 (fp16) or 17 (bf16)
// vector instructions per 8 weights and lane; at the rate HBM delivers weights that is about a third
// (two thirds) of the vector issue slots.
//
// Work split. Few rows, or few columns of a long K: a workgroup owns 16 or 32 columns, its eight waves take the 128-deep
// blocks of K in turn, straight from memory, and add their sums through LDS in wave order (w4_kernel). More
// rows: the waves share x in LDS and divide the columns, and with few columns K too (w4_rows_kernel). When
// that leaves compute units without work, K is cut over workgroups as well, into fp32 planes that a second
// kernel adds in order.
//
// Measured (weights cold, medians). 1 row of 8192 x 8192, G = 128: 10.4 us, 3.3 TB/s of 35 MB, with 5 us of them the
// launch and the first loads; 16 rows of 28672 x 8192, G = 64 with zero points: 31 us, 4.0 TB/s (a read-only stream
// 5.5); 32 rows over 8 experts of 4096 x 4096: 17.4 us, 4.0 TB/s. With many rows the unpacking bounds it, since every
// 64 rows unpack all weights again: 512 rows of 8192 x 8192, G = 128: 79 us fp16, 874 TFLOP/s, bf16 93 us. 128 rows to
// a workgroup halve that but leave registers for two waves a SIMD only (timed together, 90 and 95 us against 76 and
// 85). From about a thousand rows on, one unpacking and a dense product would be faster
// (8192 x 8192 bf16, G = 64 with zero points, 1024 rows: 178 us; the dense product takes 103).
#include "spt_device.h"
#include "spt_experts.h"

namespace spt {

// ------------------------------------------------------------------------------ layout
// Packed words: [matrix][n/16][k/128][lane][4]. Word s of lane l holds the weights of column l % 16,
// k = 32 s + 8 (l / 16) + 0 .. 7 of the block, element 2p in bits 4p and element 2p + 1 in bits
// 16 + 4p, so that one mask takes a pair to the two halves of a register. Behind them the scales
// [matrix][n/16][k/128][16][128 / G], then the zero points in the same order, a byte each.
// Columns past N and k past K hold weight 0 with scale 0.
__global__ void __launch_bounds__(256) w4_pack_kernel(W4PackArgs a) {
  const int n16 = (a.n + 15) / 16, kb = (a.k + 127) / 128;
  const int64_t words = a.matrices * n16 * kb * 256;
  unsigned* out = (unsigned*)a.packed;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < words; i += (int64_t)gridDim.x * 256) {
    const int s = (int)(i & 3), lane = (int)(i >> 2) & 63;
    const int64_t blk = i >> 8;
    const int b = (int)(blk % kb);
    const int64_t col = blk / kb;  // matrix * n16 + column block
    const int n = (int)(col % n16) * 16 + (lane & 15), k0 = b * 128 + s * 32 + 8 * (lane >> 4);
    const unsigned char* q = a.q + ((col / n16) * a.n + n) * (int64_t)a.k + k0;
    unsigned w = 0;
    if (n < a.n) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const unsigned v = k0 + e < a.k ? q[e] & 15u : 0u;
        w |= v << (4 * (e >> 1) + 16 * (e & 1));
      }
    }
    out[i] = w;
  }
}

__global__ void __launch_bounds__(256) w4_pack_groups_kernel(W4PackArgs a) {
  const int n16 = (a.n + 15) / 16, kb = (a.k + 127) / 128, gpk = 128 / a.group, groups = (a.k + a.group - 1) / a.group;
  const int64_t blocks = a.matrices * n16 * kb, total = blocks * 16 * gpk;
  unsigned short* sc = (unsigned short*)(a.packed + blocks * 1024);
  unsigned char* zp = (unsigned char*)(sc + total);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int g = (int)(i % gpk), c = (int)(i / gpk) & 15;
    const int64_t blk = i / (16 * gpk);
    const int64_t col = blk / kb;
    const int n = (int)(col % n16) * 16 + c, gr = (int)(blk % kb) * gpk + g;
    const bool in = n < a.n && gr < groups;
    const int64_t at = ((col / n16) * a.n + n) * (int64_t)groups + gr;
    sc[i] = in ? a.scales[at] : (unsigned short)0;
    if (a.zeros) zp[i] = in ? a.zeros[at] & 15 : 0;
  }
}

// ------------------------------------------------------------------------------ four bits to operands
// Eight weights minus their zero point as a matrix operand. A nibble placed in the low bits of the
// fp16 pattern of 1024 (or, shifted by four, of 64) reads 1024 + q (64 + q): two pairs come out of a
// word by a mask alone, two more after one shift. (The pattern of 1024 for this: Kim, Henry, Fahim and Hassan
// Awadalla, "Who Says Elephants Can't Run", 2022.)
struct ZeroF16 {
  unsigned c0, c1;  // -(1024 + z), -(64 + z) in both halves
};
struct ZeroF32 {
  float c0, c1;
};
__device__ __forceinline__ unsigned and_or(unsigned v, unsigned m, unsigned o) { return (v & m) | o; }
__device__ __forceinline__ unsigned add_f16x2(unsigned a, unsigned b) {
  return __builtin_bit_cast(unsigned, __builtin_bit_cast(f16x2, a) + __builtin_bit_cast(f16x2, b));
}
__device__ __forceinline__ u32x4 unpack(unsigned w, const ZeroF16& z) {
  u32x4 r;
  const unsigned v = w >> 8;
  r[0] = add_f16x2(and_or(w, 0x000F000Fu, 0x64006400u), z.c0);
  r[1] = add_f16x2(and_or(w, 0x00F000F0u, 0x54005400u), z.c1);
  r[2] = add_f16x2(and_or(v, 0x000F000Fu, 0x64006400u), z.c0);
  r[3] = add_f16x2(and_or(v, 0x00F000F0u, 0x54005400u), z.c1);
  return r;
}
// bf16 has no packed arithmetic: each half of the fp16 pair goes through one mixed-precision
// multiply-add (half * 1 + c, exact) into fp32, whose upper 16 bits are the bf16 value, exact too.
__device__ __forceinline__ unsigned minus_bf16(unsigned pair, float c) {
  float lo, hi;
  asm("v_fma_mix_f32 %0, %1, 1.0, %2 op_sel_hi:[1,0,0]" : "=v"(lo) : "v"(pair), "v"(c));
  asm("v_fma_mix_f32 %0, %1, 1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(hi) : "v"(pair), "v"(c));
  return __builtin_amdgcn_perm(__builtin_bit_cast(unsigned, hi), __builtin_bit_cast(unsigned, lo), 0x07060302u);
}
__device__ __forceinline__ u32x4 unpack(unsigned w, const ZeroF32& z) {
  u32x4 r;
  const unsigned v = w >> 8;
  r[0] = minus_bf16(and_or(w, 0x000F000Fu, 0x64006400u), z.c0);
  r[1] = minus_bf16(and_or(w, 0x00F000F0u, 0x54005400u), z.c1);
  r[2] = minus_bf16(and_or(v, 0x000F000Fu, 0x64006400u), z.c0);
  r[3] = minus_bf16(and_or(v, 0x00F000F0u, 0x54005400u), z.c1);
  return r;
}

template <int T>
__device__ __forceinline__ auto zero_of(unsigned z) {
  if constexpr (T == 1) {
    const float f = (float)z;
    return ZeroF32{-1024.f - f, -64.f - f};
  } else {
    const unsigned p = z | z << 16;
    return ZeroF16{0xE400E400u + p, 0xD400D400u + (p << 4)};
  }
}
template <int T>
__device__ __forceinline__ float scale_of(unsigned s) {
  if constexpr (T == 1) return __builtin_bit_cast(float, s << 16);
  else return (float)__builtin_bit_cast(_Float16, (unsigned short)s);
}

constexpr int kLoadNonTemporal = 2;  // cache policy: the weights are read once

// B bytes (1, 2, 4 or 8) of a lane
template <int B>
__device__ __forceinline__ auto load_groups(__amdgpu_buffer_rsrc_t r, int voff, int soff) {
  if constexpr (B == 8) return __builtin_bit_cast(uint64_t, __builtin_amdgcn_raw_buffer_load_b64(r, voff, soff, 0));
  else if constexpr (B == 4) return __builtin_amdgcn_raw_buffer_load_b32(r, voff, soff, 0);
  else if constexpr (B == 2) return __builtin_amdgcn_raw_buffer_load_b16(r, voff, soff, 0);
  else return __builtin_amdgcn_raw_buffer_load_b8(r, voff, soff, 0);
}

// The lane's chunk of eight x at byte offset voff + soff, of which `left` exist; the rest are zeros. A chunk
// that K cuts is put together from its elements, eight loads at once and no branch (one behind the other
// they made the last block take longer than all others).
__device__ __forceinline__ u32x4 load_cut(__amdgpu_buffer_rsrc_t r, unsigned voff, int soff, int left, bool whole) {
  if (whole) return __builtin_amdgcn_raw_buffer_load_b128(r, left > 0 ? voff : kOOB, soff, 0);
  unsigned v[8];
#pragma unroll
  for (int m = 0; m < 8; ++m)
    v[m] = (unsigned short)__builtin_amdgcn_raw_buffer_load_b16(r, m < left ? voff + 2 * m : kOOB, soff, 0);
  return u32x4{v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16};
}

// out: 0 fp16, 1 bf16, 2 fp32 (the same for a whole launch)
__device__ __forceinline__ void put_one(int out, char* p, int64_t i, float v) {
  if (out == 2) ((float*)p)[i] = v;
  else ((unsigned short*)p)[i] = (unsigned short)(out == 1 ? pack_bf16(v, 0.f) : pack_f16(v, 0.f));
}

// ------------------------------------------------------------------------------ the product
// T: 0 fp16, 1 bf16 (x and scales). MT, NT: 16-row and 16-column blocks. GPK: groups per 128 k.
// W waves. D: 128-deep blocks of weights in flight per wave.
template <int T, int MT, int NT, int GPK, bool ZERO, int W, int D>
__global__ void __launch_bounds__(64 * W) w4_kernel(W4Args a) {
  using TIn = std::conditional_t<T == 1, __bf16, _Float16>;
  using GroupBits = std::conditional_t<GPK == 4, uint64_t, std::conditional_t<GPK == 2, unsigned, unsigned short>>;
  using ZeroBits = std::conditional_t<GPK == 4, unsigned, std::conditional_t<GPK == 2, unsigned short, unsigned char>>;
  constexpr int BM = 16 * MT;
  __shared__ float red[W][MT * NT][256];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, h = lane >> 4;
  const int nblocks = (a.n16 + NT - 1) / NT;
  const int nb = (int)(blockIdx.x % (unsigned)nblocks) * NT, split = (int)(blockIdx.x / (unsigned)nblocks);

  int e = 0, row0 = (int)blockIdx.y * BM, rows = a.rows - row0;
  if (a.offsets) {
    const GroupBlock g = find_group(a.offsets, a.experts, a.rows, BM, 1, a.rest != 0, (int)blockIdx.y);
    if (g.e < 0) return;
    e = g.e;
    row0 = g.begin + g.block * BM;
    rows = g.end - row0;
  }
  rows = rows < BM ? rows : BM;
  const int per = (a.kb + a.splits - 1) / a.splits;
  const int kb0 = split * per, kb1 = e == a.experts && a.offsets ? kb0 : (kb0 + per < a.kb ? kb0 + per : a.kb);

  const __amdgpu_buffer_rsrc_t rx =
      make_rsrc(a.x + (int64_t)row0 * a.ldx * 2, ((uint64_t)(rows - 1) * a.ldx + a.k) * 2);
  unsigned xo[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) xo[i] = 16 * i + c < rows ? (unsigned)((16 * i + c) * (int)a.ldx + 8 * h) * 2u : kOOB;

  // The weights from this wave's first column block on. A block's offset is wave-uniform and rides in the
  // load's scalar offset: 64-bit lane addresses would cost vector instructions at every load.
  const int64_t block0 = ((int64_t)e * a.n16 + nb) * a.kb;
  const uint64_t blocks = (uint64_t)(a.n16 - nb < NT ? a.n16 - nb : NT) * a.kb;
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.w + block0 * 1024, blocks * 1024);
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(a.scales + block0 * (32 * GPK), blocks * (32 * GPK));
  const __amdgpu_buffer_rsrc_t rz = make_rsrc(a.zeros + block0 * (16 * GPK), blocks * (16 * GPK));
  // the workgroup's last columns may have fewer than NT blocks: the missing ones repeat the last
  int nstep[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) nstep[j] = (nb + j < a.n16 ? j : a.n16 - 1 - nb) * a.kb;

  // A block's loads. Loads complete in the order they were issued, so x travels in the same stage as
  // the weights it meets: loaded when needed, it would stand behind the weights of the stages to come,
  // and every block would wait for all of them.
  struct Stage {
    u32x4 q[NT];
    u32x4 x[4][MT];
    GroupBits s[NT];
    ZeroBits z[NT];
  };
  auto fetch_w = [&](Stage& st, int kb) SPT_INLINE {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int b = nstep[j] + kb;
      st.q[j] = __builtin_amdgcn_raw_buffer_load_b128(rw, lane * 16, b * 1024, kLoadNonTemporal);
      st.s[j] = load_groups<2 * GPK>(rs, c * (2 * GPK), b * (32 * GPK));
      if constexpr (ZERO) st.z[j] = (ZeroBits)load_groups<GPK>(rz, c * GPK, b * (16 * GPK));
    }
  };
  auto fetch = [&](Stage& st, int kb) SPT_INLINE {
    fetch_w(st, kb);
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < MT; ++i) st.x[s][i] = __builtin_amdgcn_raw_buffer_load_b128(rx, xo[i], 2 * (kb * 128 + s * 32), 0);
  };
  // the last block of a K that is no multiple of 128
  auto fetch_cut = [&](Stage& st, int kb) SPT_INLINE {
    fetch_w(st, kb);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int k0 = kb * 128 + s * 32;
#pragma unroll
      for (int i = 0; i < MT; ++i) st.x[s][i] = load_cut(rx, xo[i], 2 * k0, a.k - k0 - 8 * h, (a.k & 7) == 0);
    }
  };

  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  auto compute = [&](const Stage& st) SPT_INLINE {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int g = 0; g < GPK; ++g) {
        const auto z = zero_of<T>(ZERO ? (unsigned)(st.z[j] >> (8 * g)) & 0xFFu : 8u);
        f32x4 sum[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) sum[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = g * (4 / GPK); s < (g + 1) * (4 / GPK); ++s) {
          const u32x4 wf = unpack(st.q[j][s], z);
#pragma unroll
          for (int i = 0; i < MT; ++i) sum[i] = mfma16<TIn>(st.x[s][i], wf, sum[i]);
        }
        const float sc = scale_of<T>((unsigned)(st.s[j] >> (16 * g)) & 0xFFFFu);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(sum[i][r], sc, acc[i][j][r]);
      }
    }
  };

  const int kb_full = kb1 < (a.k >> 7) ? kb1 : a.k >> 7;  // blocks below it lie inside K
  // Block i of this wave is block kb0 + wave + i * W. The steady loop loads in the same order whatever
  // happens, so that a block's wait leaves the loads of the D - 1 blocks behind it in flight; the last
  // blocks, which load no more, are computed apart. (A load under a condition inside the loop makes every
  // wait a wait for all.)
  const int mine = kb_full - kb0 - wave > 0 ? (kb_full - kb0 - wave + W - 1) / W : 0;
  if (mine > 0) {
    auto at = [&](int i) SPT_INLINE { return kb0 + wave + (i < mine ? i : mine - 1) * W; };
    Stage st[D];
#pragma unroll
    for (int d = 0; d < D; ++d) {
      fetch(st[d], at(d));
      __builtin_amdgcn_sched_barrier(0);
    }
    int i = 0;
    for (; i + 2 * D <= mine; i += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        compute(st[d]);
        __builtin_amdgcn_sched_barrier(0);
        fetch(st[d], at(i + D + d));
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (i + d < mine) compute(st[d]);
      if (i + D + d < mine) fetch(st[d], at(i + D + d));
    }
#pragma unroll
    for (int d = 0; d < D - 1; ++d)
      if (i + D + d < mine) compute(st[d]);
  }
  if (kb_full < kb1 && kb_full >= kb0 && (kb_full - kb0) % W == wave) {
    Stage st;
    fetch_cut(st, kb_full);
    compute(st);
  }

  // the waves' sums, added in wave order
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) *(f32x4*)&red[wave][i * NT + j][4 * lane] = acc[i][j];
  __syncthreads();
  // consecutive threads take consecutive columns
  for (int t = threadIdx.x; t < MT * NT * 256; t += 64 * W) {
    const int n_in = t % (16 * NT), m = t / (16 * NT);
    const int j = n_in >> 4, i = m >> 4, src = 4 * ((n_in & 15) + 16 * ((m & 15) >> 2)) + (m & 3);
    const int n = nb * 16 + n_in;
    if (m >= rows || n >= a.n) continue;
    float v = red[0][i * NT + j][src];
#pragma unroll
    for (int w = 1; w < W; ++w) v += red[w][i * NT + j][src];
    if (a.splits > 1) ((float*)a.out)[split * a.plane + (int64_t)(row0 + m) * a.n + n] = v;
    else put_one(a.out_dtype, a.out, (int64_t)(row0 + m) * a.ldo + n, v);
  }
}

// The same product with more rows: the waves of a workgroup split its columns (WN) and the blocks of K
// (WK), and share x. An x fragment costs as much of the load path as a wave's whole block of weights, so
// each is loaded once for WN waves, a block ahead, into registers and from there into one of two LDS
// buffers, in the order the matrix instruction wants it (lane-contiguous, no bank conflicts).
template <int T, int MT, int NT, int WN, int WK, int GPK, bool ZERO>
__global__ void __launch_bounds__(64 * WN * WK) w4_rows_kernel(W4Args a) {
  using TIn = std::conditional_t<T == 1, __bf16, _Float16>;
  using GroupBits = std::conditional_t<GPK == 4, uint64_t, std::conditional_t<GPK == 2, unsigned, unsigned short>>;
  using ZeroBits = std::conditional_t<GPK == 4, unsigned, std::conditional_t<GPK == 2, unsigned short, unsigned char>>;
  constexpr int BM = 16 * MT, W = WN * WK;
  constexpr int NX = 4 * MT / WN;  // x fragments a wave loads per block
  constexpr int XBUF = WK * 4 * MT * 1024, RED = W * MT * NT * 1024;
  static_assert(4 * MT % WN == 0, "the waves of a block load the same number of fragments");
  __shared__ __attribute__((aligned(16))) char lds[2 * XBUF > RED ? 2 * XBUF : RED];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wk = wave / WN, wn = wave % WN;
  const int c = lane & 15, h = lane >> 4;
  const int nblocks = (a.n16 + NT * WN - 1) / (NT * WN);
  const int col16 = (int)(blockIdx.x % (unsigned)nblocks) * (NT * WN), split = (int)(blockIdx.x / (unsigned)nblocks);
  const int nb = col16 + wn * NT < a.n16 ? col16 + wn * NT : a.n16 - 1;  // this wave's first column block

  int e = 0, row0 = (int)blockIdx.y * BM, rows = a.rows - row0;
  if (a.offsets) {
    const GroupBlock g = find_group(a.offsets, a.experts, a.rows, BM, 1, a.rest != 0, (int)blockIdx.y);
    if (g.e < 0) return;
    e = g.e;
    row0 = g.begin + g.block * BM;
    rows = g.end - row0;
  }
  rows = rows < BM ? rows : BM;
  const bool none = a.offsets && e == a.experts;  // rows of nobody: zeros
  const int per = (a.kb + a.splits - 1) / a.splits;
  const int kb0 = split * per, kb1 = none ? kb0 : (kb0 + per < a.kb ? kb0 + per : a.kb);
  const int kb_full = kb1 < (a.k >> 7) ? kb1 : a.k >> 7;

  const __amdgpu_buffer_rsrc_t rx =
      make_rsrc(a.x + (int64_t)row0 * a.ldx * 2, ((uint64_t)(rows - 1) * a.ldx + a.k) * 2);
  // fragment i of this wave: matrix step f / MT, rows 16 (f % MT) .., f = wn * NX + i
  unsigned xo[NX];
#pragma unroll
  for (int i = 0; i < NX; ++i) {
    const int f = wn * NX + i, m = 16 * (f % MT) + c;
    xo[i] = m < rows ? (unsigned)(m * (int)a.ldx + 32 * (f / MT) + 8 * h) * 2u : kOOB;
  }
  auto x_at = [&](int buf, int w, int f) SPT_INLINE { return lds + buf * XBUF + (w * 4 * MT + f) * 1024 + 16 * lane; };

  // The weights from this wave's first column block on. A block's offset is wave-uniform and rides in the
  // load's scalar offset: 64-bit lane addresses would cost vector instructions at every load.
  const int64_t block0 = ((int64_t)e * a.n16 + nb) * a.kb;
  const uint64_t blocks = (uint64_t)(a.n16 - nb < NT ? a.n16 - nb : NT) * a.kb;
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.w + block0 * 1024, blocks * 1024);
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(a.scales + block0 * (32 * GPK), blocks * (32 * GPK));
  const __amdgpu_buffer_rsrc_t rz = make_rsrc(a.zeros + block0 * (16 * GPK), blocks * (16 * GPK));
  int nstep[NT];  // column blocks past the last repeat it
#pragma unroll
  for (int j = 0; j < NT; ++j) nstep[j] = (nb + j < a.n16 ? j : a.n16 - 1 - nb) * a.kb;

  struct Stage {
    u32x4 q[NT];
    GroupBits s[NT];
    ZeroBits z[NT];
  };
  auto fetch_w = [&](Stage& st, int kb) SPT_INLINE {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int b = nstep[j] + kb;
      st.q[j] = __builtin_amdgcn_raw_buffer_load_b128(rw, lane * 16, b * 1024, kLoadNonTemporal);
      st.s[j] = load_groups<2 * GPK>(rs, c * (2 * GPK), b * (32 * GPK));
      if constexpr (ZERO) st.z[j] = (ZeroBits)load_groups<GPK>(rz, c * GPK, b * (16 * GPK));
    }
  };

  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // one block of weights with x from LDS buffer `buf`
  auto compute = [&](const Stage& st, int buf, int w) SPT_INLINE {
#pragma unroll
    for (int g = 0; g < GPK; ++g) {
      constexpr int SPG = 4 / GPK;  // matrix steps per group
      decltype(zero_of<T>(0u)) z[NT];
      f32x4 sum[NT][MT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        z[j] = zero_of<T>(ZERO ? (unsigned)(st.z[j] >> (8 * g)) & 0xFFu : 8u);
#pragma unroll
        for (int i = 0; i < MT; ++i) sum[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int s = 0; s < SPG; ++s) {
        u32x4 xf[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) xf[i] = *(const u32x4*)x_at(buf, w, (g * SPG + s) * MT + i);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const u32x4 wf = unpack(st.q[j][g * SPG + s], z[j]);
#pragma unroll
          for (int i = 0; i < MT; ++i) sum[j][i] = mfma16<TIn>(xf[i], wf, sum[j][i]);
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const float sc = scale_of<T>((unsigned)(st.s[j] >> (16 * g)) & 0xFFFFu);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(sum[j][i][r], sc, acc[i][j][r]);
      }
    }
  };

  const int n = kb_full - kb0 > 0 ? (kb_full - kb0 + WK - 1) / WK : 0;  // rounds of WK blocks
  if (n > 0) {
    // past the end: the last block again, loaded and not used, so that every round issues the same loads
    auto block = [&](int i) SPT_INLINE {
      const int b = kb0 + i * WK + wk;
      return b < kb_full ? b : kb_full - 1;
    };
    u32x4 xs[NX];
    auto fetch_x = [&](int i) SPT_INLINE {
#pragma unroll
      for (int f = 0; f < NX; ++f) xs[f] = __builtin_amdgcn_raw_buffer_load_b128(rx, xo[f], 2 * 128 * block(i), 0);
    };
    auto put_x = [&](int buf) SPT_INLINE {
#pragma unroll
      for (int f = 0; f < NX; ++f) *(u32x4*)x_at(buf, wk, wn * NX + f) = xs[f];
    };
    Stage st[2];
    fetch_x(0);
    fetch_w(st[0], block(0));
    __builtin_amdgcn_sched_barrier(0);
    put_x(0);
    fetch_x(1);
    fetch_w(st[1], block(1));
    wait_lgkmcnt0();
    barrier_sync();
    for (int i = 0; i < n; i += 2) {
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        put_x(d ^ 1);  // round i + d + 1; its buffer was read in the round before this one
        __builtin_amdgcn_sched_barrier(0);
        fetch_x(i + d + 2);
        __builtin_amdgcn_sched_barrier(0);
        if (kb0 + (i + d) * WK + wk < kb_full) compute(st[d], d, wk);
        __builtin_amdgcn_sched_barrier(0);
        fetch_w(st[d], block(i + d + 2));
        wait_lgkmcnt0();
        barrier_sync();
      }
    }
  }
  if (kb_full < kb1 && kb_full >= kb0) {
    // the last block of a K that is no multiple of 128, for the waves of K part 0
    Stage st;
    fetch_w(st, kb_full);
    barrier_sync();
    if (wk == 0) {
#pragma unroll
      for (int f = 0; f < NX; ++f) {
        const int left = a.k - kb_full * 128 - 32 * ((wn * NX + f) / MT) - 8 * h;
        const u32x4 r = load_cut(rx, xo[f], 2 * 128 * kb_full, left, (a.k & 7) == 0);
        *(u32x4*)x_at(0, 0, wn * NX + f) = r;
      }
    }
    wait_lgkmcnt0();
    barrier_sync();
    if (wk == 0) compute(st, 0, 0);
  }

  // the K parts' sums, added in their order; consecutive threads take consecutive columns
  wait_lgkmcnt0();
  barrier_sync();  // the buffers have been read
  float* red = (float*)lds;
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) *(f32x4*)&red[((wk * MT + i) * WN * NT + wn * NT + j) * 256 + 4 * lane] = acc[i][j];
  __syncthreads();
  constexpr int COLS = 16 * NT * WN;
  for (int t = threadIdx.x; t < BM * COLS; t += 64 * W) {
    const int n_in = t % COLS, m = t / COLS;
    const int col = col16 * 16 + n_in;
    if (m >= rows || col >= a.n) continue;
    const int at = ((m >> 4) * WN * NT + (n_in >> 4)) * 256 + 4 * ((n_in & 15) + 16 * ((m & 15) >> 2)) + (m & 3);
    float v = red[at];
#pragma unroll
    for (int w = 1; w < WK; ++w) v += red[at + w * MT * WN * NT * 256];
    if (a.splits > 1) ((float*)a.out)[split * a.plane + (int64_t)(row0 + m) * a.n + col] = v;
    else put_one(a.out_dtype, a.out, (int64_t)(row0 + m) * a.ldo + col, v);
  }
}

// out = the planes of a cut sum (of these products or the grouped ones) added in order, rounded once. With
// offsets, rows that belong to no expert are left alone.
__global__ void __launch_bounds__(256) add_planes_kernel(PlaneArgs r) {
  const int first = r.offsets ? clampi(r.offsets[0], 0, r.rows) : 0;
  const int last = r.offsets ? clampi(r.offsets[r.experts], 0, r.rows) : r.rows;
  const int64_t end = (int64_t)last * r.n;
  for (int64_t i = (int64_t)first * r.n + (int64_t)blockIdx.x * 256 + threadIdx.x; i < end; i += (int64_t)gridDim.x * 256) {
    float v = r.parts[i];
    for (int s = 1; s < r.splits; ++s) v += r.parts[s * r.plane + i];
    const int64_t row = i / r.n;
    put_one(r.out_dtype, r.out, row * r.ldo + (i - row * r.n), v);
  }
}

// ------------------------------------------------------------------------------ instantiations
template <int T, int MT, int NT, int W, int D>
static W4Entry w4_pick_group(int gpk, bool zero) {
  W4Entry e{nullptr, MT, NT, W, W};
  if (gpk == 1) e.fn = zero ? (const void*)&w4_kernel<T, MT, NT, 1, true, W, D> : (const void*)&w4_kernel<T, MT, NT, 1, false, W, D>;
  else if (gpk == 2) e.fn = zero ? (const void*)&w4_kernel<T, MT, NT, 2, true, W, D> : (const void*)&w4_kernel<T, MT, NT, 2, false, W, D>;
  else e.fn = zero ? (const void*)&w4_kernel<T, MT, NT, 4, true, W, D> : (const void*)&w4_kernel<T, MT, NT, 4, false, W, D>;
  return e;
}
template <int T, int MT, int NT, int WN, int WK>
static W4Entry w4_pick_rows(int gpk, bool zero) {
  W4Entry e{nullptr, MT, NT * WN, WN * WK, WK};
  if (gpk == 1) e.fn = zero ? (const void*)&w4_rows_kernel<T, MT, NT, WN, WK, 1, true> : (const void*)&w4_rows_kernel<T, MT, NT, WN, WK, 1, false>;
  else if (gpk == 2) e.fn = zero ? (const void*)&w4_rows_kernel<T, MT, NT, WN, WK, 2, true> : (const void*)&w4_rows_kernel<T, MT, NT, WN, WK, 2, false>;
  else e.fn = zero ? (const void*)&w4_rows_kernel<T, MT, NT, WN, WK, 4, true> : (const void*)&w4_rows_kernel<T, MT, NT, WN, WK, 4, false>;
  return e;
}
template <int T>
static W4Entry w4_pick(int variant, int gpk, bool zero) {
  switch (variant) {
    case 0: return w4_pick_group<T, 1, 1, 8, 4>(gpk, zero);
    case 1: return w4_pick_group<T, 1, 2, 8, 2>(gpk, zero);
    case 2: return w4_pick_rows<T, 1, 1, 4, 4>(gpk, zero);
    case 3: return w4_pick_rows<T, 2, 1, 4, 4>(gpk, zero);
    case 4: return w4_pick_rows<T, 2, 2, 4, 2>(gpk, zero);
    case 5: return w4_pick_rows<T, 4, 1, 8, 1>(gpk, zero);
    case 6: return w4_pick_rows<T, 4, 2, 8, 1>(gpk, zero);
    default: return w4_pick_rows<T, 1, 2, 4, 2>(gpk, zero);
  }
}
W4Entry w4_entry(int variant, int bf16, int gpk, bool zero) {
  return bf16 ? w4_pick<1>(variant, gpk, zero) : w4_pick<0>(variant, gpk, zero);
}
const void* w4_pack_fn() { return (const void*)&w4_pack_kernel; }
const void* w4_pack_groups_fn() { return (const void*)&w4_pack_groups_kernel; }
const void* add_planes_fn() { return (const void*)&add_planes_kernel; }

}  // namespace spt
