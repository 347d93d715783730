// Products of microscaled operands with few rows: what bounds them is reading B once.
//
// A workgroup has up to 16 MT rows and 16 NF columns (NF = 1: over 172 shapes 32 columns took 21 % longer and 64 50 %, for
// want of workgroups), and its eight waves share out k: each streams its k-steps of B (and of A, which lies in the L2) from
// memory to registers in the matrix instruction's own order, with no LDS on the way, several k-steps of it in flight. The
// waves' sums meet in LDS once at the end. Row r of fragment f is operand row MT r + f: a lane's MT scale bytes are
// neighbours, one load that the instruction's operand select takes apart. 32 rows of 4096 x 4096 8 x 4: 8.8 us, the tile kernel in
// four parts 9.2; where there are more columns than compute units have workgroups, it loses (6144 x 4096: 15.8 against 9.9).
//   B goes by with the non-temporal hint: nobody reads it again.
#include "spt_mx_device.h"

namespace spt {

constexpr int kSkinnyWaves = 8;

// N bytes (1, 2, 4) as a word.
template <int N>
__device__ __forceinline__ unsigned load_bytes(__amdgpu_buffer_rsrc_t r, unsigned voffset, unsigned soffset) {
  if constexpr (N == 1) return (unsigned)(unsigned char)__builtin_amdgcn_raw_buffer_load_b8(r, voffset, soffset, 0);
  else if constexpr (N == 2) return (unsigned)(unsigned short)__builtin_amdgcn_raw_buffer_load_b16(r, voffset, soffset, 0);
  else return (unsigned)__builtin_amdgcn_raw_buffer_load_b32(r, voffset, soffset, 0);
}

template <int FA, int FB, bool EXACT, int MT>
__global__ void __launch_bounds__(64 * kSkinnyWaves) mx_skinny_kernel(MxGemmArgs args) {
  constexpr int W = kSkinnyWaves, NF = 1;
  // Pieces (k-steps) in flight: what about 128 registers hold, 2 to 8.
  constexpr int REGS = MT * FA + NF * FB + 2, D = 128 / REGS < 2 ? 2 : 128 / REGS > 8 ? 8 : 128 / REGS;
  __shared__ float red[W][MT * NF * 4][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q4 = lane >> 4;
  const int col0 = blockIdx.x * (16 * NF);
  const int lda = args.blocks * (4 * FA), ldb = args.blocks * (4 * FB);
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(args.a, (uint64_t)args.m * lda);
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(args.b + (int64_t)col0 * ldb, (uint64_t)(args.n - col0) * ldb);
  const int sbytes = args.blocks * kMxScaleRows;  // of 64 rows; a workgroup's columns lie inside 64
  const __amdgpu_buffer_rsrc_t rsa = make_rsrc(args.as, (uint64_t)sbytes);
  const __amdgpu_buffer_rsrc_t rsb = make_rsrc(args.bs + (int64_t)(col0 / 64) * sbytes, (uint64_t)sbytes);

  const unsigned in_row = EXACT ? 32u * q4 : 16u * q4;  // of a k-step: this lane's first chunk
  constexpr unsigned kSecond = EXACT ? 16u : 64u;       // from there to its second, in 8 bits
  const unsigned a_in = FA == 8 ? in_row : 16u * q4, b_in = FB == 8 ? in_row : 16u * q4;
  unsigned va[MT], vb[NF];
#pragma unroll
  for (int f = 0; f < MT; ++f) va[f] = (unsigned)((MT * r16 + f) * lda) + a_in;
#pragma unroll
  for (int f = 0; f < NF; ++f) vb[f] = (unsigned)((NF * r16 + f) * ldb) + b_in;
  const unsigned vsa = (unsigned)(q4 * 64 + MT * r16), vsb = (unsigned)(q4 * 64 + (col0 & 63) + NF * r16);

  struct Piece {
    u32x4 a[MT][FA / 4], b[NF][FB / 4];
    unsigned sa, sb;
  };
  const int ks1 = args.ksteps;
  auto load = [&](Piece& p, int ks) SPT_INLINE {
    const unsigned past = ks < ks1 ? 0u : kOOB;  // set, it moves an offset beyond the descriptor's end
    const unsigned ka = (unsigned)(ks * (16 * FA)), kb = (unsigned)(ks * (16 * FB)), kc = (unsigned)(ks * 256);
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const unsigned v = vb[f] | past;
      p.b[f][0] = __builtin_amdgcn_raw_buffer_load_b128(rb, v, kb, 2);
      if constexpr (FB == 8) p.b[f][1] = __builtin_amdgcn_raw_buffer_load_b128(rb, v + kSecond, kb, 2);
    }
    p.sb = load_bytes<NF>(rsb, vsb | past, kc);
#pragma unroll
    for (int f = 0; f < MT; ++f) {
      const unsigned v = va[f] | past;
      p.a[f][0] = __builtin_amdgcn_raw_buffer_load_b128(ra, v, ka, 0);
      if constexpr (FA == 8) p.a[f][1] = __builtin_amdgcn_raw_buffer_load_b128(ra, v + kSecond, ka, 0);
    }
    p.sa = load_bytes<MT>(rsa, vsa | past, kc);
  };
  f32x4 acc[MT][NF];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](const Piece& p) SPT_INLINE {
    if constexpr (EXACT) {
      static_for<4>([&](auto p_c) SPT_INLINE {
        constexpr int h = decltype(p_c)::value;
        u32x4 xb[MT], yb[NF];
        static_for<MT>([&](auto f_c) SPT_INLINE {
          constexpr int f = decltype(f_c)::value;
          xb[f] = mx_bf16<FA, h>(p.a[f][0], p.a[f][FA / 4 - 1], (p.sa >> (8 * f)) & 255u);
        });
        static_for<NF>([&](auto f_c) SPT_INLINE {
          constexpr int f = decltype(f_c)::value;
          yb[f] = mx_bf16<FB, h>(p.b[f][0], p.b[f][FB / 4 - 1], (p.sb >> (8 * f)) & 255u);
        });
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < NF; ++j) acc[i][j] = mfma16<__bf16>(xb[i], yb[j], acc[i][j]);
      });
    } else {
      i32x8 x[MT], y[NF];
#pragma unroll
      for (int f = 0; f < MT; ++f) x[f] = mx_operand<FA>(p.a[f][0], p.a[f][FA / 4 - 1]);
#pragma unroll
      for (int f = 0; f < NF; ++f) y[f] = mx_operand<FB>(p.b[f][0], p.b[f][FB / 4 - 1]);
      static_for<MT * NF>([&](auto m_c) SPT_INLINE {
        constexpr int i = decltype(m_c)::value / NF, j = decltype(m_c)::value % NF;
        acc[i][j] = mfma_mx<FA, FB, i, j>(x[i], y[j], acc[i][j], p.sa, p.sb);
      });
    }
  };

  // Pieces wave, wave + W, ..: neighbouring waves read neighbouring parts of a row's lines. One past the end reads zeros.
  unsigned far = 0;
  {
    Piece p[D];
    int ks = wave;
#pragma unroll
    for (int d = 0; d < D; ++d) load(p[d], ks + d * W);
    for (; ks < ks1; ks += D * W) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if constexpr (EXACT) far |= mx_far<FA, MT>(p[d].a, p[d].sa) | mx_far<FB, NF>(p[d].b, p[d].sb);
        compute(p[d]);
        __builtin_amdgcn_sched_barrier(0);  // loads moved up to here would need registers of their own
        load(p[d], ks + (D + d) * W);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  // With a far block the wave's sum is taken again, one piece at a time: mx_far_products in each of the D places above, which a branch
  // jumps over, would cost every call 1.3 us (1 x 4096^2 8 x 8: 8.1 us, 9.4).
  if constexpr (EXACT) {
    if (__builtin_expect(__any(far != 0), 0)) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int ks = wave; ks < ks1; ks += W) {
        Piece p;
        load(p, ks);
        if (__any((mx_far<FA, MT>(p.a, p.sa) | mx_far<FB, NF>(p.b, p.sb)) != 0)) mx_far_products<FA, FB, MT, NF>(p.a, p.b, p.sa, p.sb, acc);
        else compute(p);
      }
    }
  }

#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[wave][(i * NF + j) * 4 + e][lane] = acc[i][j][e];
  __syncthreads();

  // An item is one lane's NF neighbouring columns of row MT (4 q4 + e) + f, the waves' sums added in their order.
  char* out = args.c;
  for (int t = threadIdx.x; t < MT * 256; t += 64 * W) {
    const int l = t & 63, e = (t >> 6) & 3, f = t >> 8;
    const int row = MT * (4 * (l >> 4) + e) + f, col = col0 + NF * (l & 15);
    if (row >= args.m || col >= args.n) continue;
    float v[NF];
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      v[j] = red[0][(f * NF + j) * 4 + e][l];
#pragma unroll
      for (int w = 1; w < W; ++w) v[j] += red[w][(f * NF + j) * 4 + e][l];
    }
    const int64_t at = row * args.ldc + col;
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      if (col + j >= args.n) break;
      if (args.out_dtype == 2) ((float*)out)[at + j] = v[j];
      else ((unsigned short*)out)[at + j] = (unsigned short)((args.out_dtype == 1 ? pack_bf16(v[j], 0.f) : pack_f16(v[j], 0.f)) & 0xFFFFu);
    }
  }
}

template <int FA, int FB, bool EXACT>
static const void* skinny_pick(int mt) {
  return mt == 1 ? (const void*)&mx_skinny_kernel<FA, FB, EXACT, 1> : (const void*)&mx_skinny_kernel<FA, FB, EXACT, 2>;
}
MxEntry mx_skinny_entry(int fa, int fb, bool exact, int mt) {
  MxEntry e{nullptr, 16 * mt, 16, 64 * kSkinnyWaves, 1};
  if (fa == 4) e.fn = skinny_pick<4, 4, false>(mt);
  else if (fb == 4) e.fn = exact ? skinny_pick<8, 4, true>(mt) : skinny_pick<8, 4, false>(mt);
  else e.fn = exact ? skinny_pick<8, 8, true>(mt) : skinny_pick<8, 8, false>(mt);
  return e;
}

}  // namespace spt
