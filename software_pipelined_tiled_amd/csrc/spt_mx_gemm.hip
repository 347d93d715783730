// Products of microscaled operands in tiles of 32, 64 or 128 rows by 128 columns: C = A . B^T through a ring of LDS stages.
//
// Four waves, 2 x 2, of 16 FM x 64 outputs each (FM = 1, 2, 4): FM x 4 blocks of v_mfma_scale_f32_16x16x128_f8f6f4. A K-tile is
// 128 values of k, 256 where both operands have 4 bits, so that its rows are 128 bytes of each operand (64 of a 4-bit
// one beside an 8-bit one). The layout in LDS is the dense kernels': rows of eight (four) 16-byte chunks, chunk c of row r
// at c XOR (r mod 8) (at c XOR ((r / 2) mod 4) in 64-byte rows), which the direct global->LDS loads make by choosing each lane's
// source. Two workgroups to a compute unit with half of its LDS each, so that one's products hide the other's reads and
// waits (1024 x 8192^2 8 x 8: 75 us, 91 with one and twice the stages; 51 x 9280 x 1152 8 x 4, 32 rows: 6 us against 8).
//
// Rows are staged permuted: row r of fragment f is row 4r + f of the wave's 64 B rows (FM r + f of its A rows). A lane's fragments
// are then neighbouring rows, whose scales of one block are one aligned word in memory (hence scales in blocks of
// 64 rows); the instruction's operand select picks the fragment's byte, so no instruction unpacks scales. And a
// lane's results are four neighbouring columns, a quarter-wave's 128 bytes or more of a row.
//
// EXACT (8-bit operands with fp32 results): a lane reads both chunks of one 32-block instead, converts them to bf16 with
// their scale, and runs four 16x16x32 bf16 instructions, whose sums lose nothing. A wave that meets a scale which carries its values out
// of bf16's range takes that k-step in pieces (mx_far_products); looking for such scales costs up to 3 % (300 x 8192^2 8 x 8: 70 us, 69;
// 128 x 5000 x 6000 22.6, 21.9).
//
// Scales go through LDS too (1 KiB a stage; 2 with 256 values of k): each wave loads those of one 64-row block.
//   What bounds it: with few rows reading B (16 rows of 28672 x 8192 8 x 4: 30 us with part of B in the last cache, 35 from memory, 24 at
// the rate of a large copy), else its K-tiles' latency and reads (256, 512, 1024 rows of 8192^2 8 x 8: 36, 55 and 78 us; 15, 16 and 32 at
// the instruction's rate); the exact form the conversions (301 x 1025 x 8190 8 x 8: 19 us and 4 for the planes' sum, with bf16 results
// 16 in all; 8192^3 965, where the two-group kernel takes 364 for bf16 results).
#include "spt_mx_device.h"

namespace spt {

template <int F, int KS>
constexpr int mx_lds_row() { return F == 8 || KS == 2 ? 128 : 64; }

template <int FA, int FB, bool EXACT, int FM>
__global__ void __launch_bounds__(256, 2) mx_tile_kernel(MxGemmArgs args) {
  constexpr int KS = FA == 4 && FB == 4 ? 2 : 1;  // k-steps of a K-tile
  constexpr int RA = mx_lds_row<FA, KS>(), RB = mx_lds_row<FB, KS>();
  constexpr int BM = 32 * FM, A_BYTES = BM * RA, B_BYTES = 128 * RB, SC = KS * 256;  // SC: scales of 64 rows
  constexpr int STAGE = A_BYTES + B_BYTES + 4 * SC;
  constexpr int S = 80 * 1024 / STAGE;  // stages: two workgroups share a compute unit's LDS
  constexpr int LA = A_BYTES / 4096, LB = B_BYTES / 4096, LW = LA + LB + 1;  // loads of a wave
  static_assert(S >= 2 && LW * (S - 1) < 64, "ring");
  __shared__ __attribute__((aligned(1024))) char smem[S * STAGE];
  const unsigned smem_base = lds_addr(smem);

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int r16 = lane & 15, q4 = lane >> 4;
  int tm, tn, part;
  unit_decode(xcd_remap(blockIdx.x, args.grid), args.tiles_m, args.tiles_n, args.group_m, tm, tn, part);
  const int row0 = tm * BM, col0 = tn * 128;
  const int kt0 = part * args.per, kts = (args.ksteps + KS - 1) / KS;
  const int kt1 = kt0 + args.per < kts ? kt0 + args.per : kts;

  // Rows past the operand's last lie at or beyond the descriptor's end and read zero.
  const int64_t rba = (int64_t)args.blocks * (4 * FA), rbb = (int64_t)args.blocks * (4 * FB);
  const int lda = (int)rba, ldb = (int)rbb;
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(args.a + row0 * rba, (uint64_t)(args.m - row0) * rba);
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(args.b + col0 * rbb, (uint64_t)(args.n - col0) * rbb);
  const int sbytes = args.blocks * kMxScaleRows;  // of 64 rows
  const bool for_a = wave < 2;                    // whose scales this wave loads (with one block of A wave 1's are not read)
  const int sblock = (for_a ? row0 : col0) / 64 + (wave & 1);
  const int sblocks = ((for_a ? args.m : args.n) + 63) / 64;
  const __amdgpu_buffer_rsrc_t rs =
      make_rsrc((for_a ? args.as : args.bs) + (int64_t)sblock * sbytes, sblock < sblocks ? (uint64_t)sbytes : 0);

  // This lane's source in a load instruction of 1 KiB: instruction i fills LDS rows 8i .. 8i + 7 (128-byte rows) or
  // 16i .. 16i + 15; the row splits into a part of the lane and one of the instruction. fr: fragments of a wave.
  auto lane_src = [&](int rowbytes, int ld, int fr, unsigned& off, int& kbyte) SPT_INLINE {
    const int row = fr * (rowbytes == 128 ? lane >> 3 : lane >> 2);
    const int chunk = rowbytes == 128 ? (lane & 7) ^ (lane >> 3) : (lane & 3) ^ ((lane >> 3) & 3);
    kbyte = chunk * 16;
    off = (unsigned)(row * ld) + (unsigned)kbyte;
  };
  auto instr_row = [&](int rowbytes, int fr, int i) SPT_INLINE {
    return rowbytes == 128 ? 16 * fr * (i / (2 * fr)) + 8 * fr * (i & 1) + (i >> 1) % fr : 16 * fr * (i / fr) + i % fr;
  };
  unsigned a_off, b_off;
  int a_kb, b_kb;
  lane_src(RA, lda, FM, a_off, a_kb);
  lane_src(RB, ldb, 4, b_off, b_kb);

  auto issue = [&](int kt, int slot) SPT_INLINE {
    const bool real = kt < kt1;
    const unsigned base = smem_base + (unsigned)(slot * STAGE);
    const int ka = kt * (KS * 16 * FA), kb = kt * (KS * 16 * FB);  // a k-step is 16 F bytes of a row
    // with 256 values a K-tile the row's end may lie inside
    const unsigned va = real && (KS == 1 || ka + a_kb < lda) ? a_off : kOOB;
    const unsigned vb = real && (KS == 1 || kb + b_kb < ldb) ? b_off : kOOB;
#pragma unroll
    for (int j = 0; j < LA; ++j) {
      const int i = LA * wave + j;
      dma16_unseen(ra, base + i * 1024, va == kOOB ? kOOB : va + (unsigned)(instr_row(RA, FM, i) * lda), (unsigned)ka);
    }
#pragma unroll
    for (int j = 0; j < LB; ++j) {
      const int i = LB * wave + j;
      dma16_unseen(rb, base + A_BYTES + i * 1024, vb == kOOB ? kOOB : vb + (unsigned)(instr_row(RB, 4, i) * ldb), (unsigned)kb);
    }
    // 64 rows by 4 KS blocks lie together: 256 KS bytes by a quarter or half of the lanes
    if (lane < 16 * KS) {
      const int at = kt * (KS * 256) + lane * 16;
      dma16_unseen(rs, base + A_BYTES + B_BYTES + wave * SC, real && at < sbytes ? (unsigned)at : kOOB, 0);
    }
  };

  // EXACT: 0x7F in the scale bytes of rows that are not there (theirs are 0, a far one) and where a lane has fewer than four
  unsigned near_a = 0, near_b = 0;
  if constexpr (EXACT) {
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      if (f >= FM || row0 + 16 * FM * wm + FM * r16 + f >= args.m) near_a |= 0x7Fu << (8 * f);
      if (col0 + 64 * wn + 4 * r16 + f >= args.n) near_b |= 0x7Fu << (8 * f);
    }
  }
  f32x4 acc[FM][4];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // Chunk `c` of fragment f's row, operand rows at `p`.
  auto chunk = [&](const char* p, int rowbytes, int f, int c) SPT_INLINE {
    const int row = 16 * f + r16;
    const int at = rowbytes == 128 ? row * 128 + ((c ^ (r16 & 7)) << 4) : row * 64 + ((c ^ ((r16 >> 1) & 3)) << 4);
    return *(const u32x4*)(p + at);
  };
  // This lane's scale bytes of a k-step, as `compute` takes them. EXACT looks at them first, and has them read before the loads go out.
  struct Words {
    unsigned a, b;
  };
  auto scale_words = [&](const char* st) SPT_INLINE {
    const int arow = (row0 & 63) + wm * 16 * FM;
    const char* sa = st + A_BYTES + B_BYTES + (arow >> 6) * SC + (arow & 63) + FM * r16;
    const char* sb = st + A_BYTES + B_BYTES + (2 + wn) * SC;
    Words w;
    w.a = FM == 4 ? *(const unsigned*)(sa + q4 * 64) : FM == 2 ? *(const unsigned short*)(sa + q4 * 64) : *(const unsigned char*)(sa + q4 * 64);
    w.b = *(const unsigned*)(sb + q4 * 64 + 4 * r16);
    return w;
  };
  auto compute = [&](int slot, const Words& early) SPT_INLINE {
    const char* st = smem + opaque_s32(slot * STAGE);
    const char* pa = st + wm * 16 * FM * RA;
    const char* pb = st + A_BYTES + wn * 64 * RB;
    const int arow = (row0 & 63) + wm * 16 * FM;
    const char* sa = st + A_BYTES + B_BYTES + (arow >> 6) * SC + (arow & 63) + FM * r16;
    const char* sb = st + A_BYTES + B_BYTES + (2 + wn) * SC;
    static_for<KS>([&](auto s_c) SPT_INLINE {
      constexpr int s = decltype(s_c)::value;
      const unsigned wa = EXACT ? early.a : FM == 4 ? *(const unsigned*)(sa + (4 * s + q4) * 64) : FM == 2 ? *(const unsigned short*)(sa + (4 * s + q4) * 64) : *(const unsigned char*)(sa + (4 * s + q4) * 64);
      const unsigned wb = EXACT ? early.b : *(const unsigned*)(sb + (4 * s + q4) * 64 + 4 * r16);
      constexpr int CA = FA / 4, CB = FB / 4;  // chunks of a lane
      u32x4 x[FM][CA], y[4][CB];
#pragma unroll
      for (int f = 0; f < 4; ++f)
#pragma unroll
        for (int h = 0; h < CB; ++h) y[f][h] = chunk(pb, RB, f, FB == 4 ? 4 * s + q4 : EXACT ? 2 * q4 + h : q4 + 4 * h);
#pragma unroll
      for (int f = 0; f < FM; ++f)
#pragma unroll
        for (int h = 0; h < CA; ++h) x[f][h] = chunk(pa, RA, f, FA == 4 ? 4 * s + q4 : EXACT ? 2 * q4 + h : q4 + 4 * h);
      if constexpr (EXACT) {
        static_for<4>([&](auto p_c) SPT_INLINE {
          constexpr int p = decltype(p_c)::value;
          u32x4 xb[FM], yb[4];
          static_for<4>([&](auto f_c) SPT_INLINE {
            constexpr int f = decltype(f_c)::value;
            yb[f] = mx_bf16<FB, p>(y[f][0], y[f][CB - 1], (wb >> (8 * f)) & 255u);
            if constexpr (f < FM) xb[f] = mx_bf16<FA, p>(x[f][0], x[f][CA - 1], (wa >> (8 * f)) & 255u);
          });
#pragma unroll
          for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = mfma16<__bf16>(xb[i], yb[j], acc[i][j]);
        });
      } else {
        static_for<4 * FM>([&](auto m_c) SPT_INLINE {
          constexpr int i = decltype(m_c)::value / 4, j = decltype(m_c)::value % 4;
          acc[i][j] = mfma_mx<FA, FB, i, j>(mx_operand<FA>(x[i][0], x[i][CA - 1]), mx_operand<FB>(y[j][0], y[j][CB - 1]), acc[i][j], wa, wb);
        });
      }
    });
  };
  // EXACT: whether the k-step has a far block of this wave's rows; then its products are done here.
  auto far_step = [&](int slot, const Words& w) SPT_INLINE {
    if (__builtin_expect(!__any(mx_wide(w.a | near_a, w.b | near_b)), 1)) return false;
    const char* st = smem + opaque_s32(slot * STAGE);
    u32x4 x[FM][FA / 4], y[4][FB / 4];
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int h = 0; h < FB / 4; ++h) y[f][h] = chunk(st + A_BYTES + wn * 64 * RB, RB, f, FB == 4 ? q4 : 2 * q4 + h);
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
      for (int h = 0; h < FA / 4; ++h) x[f][h] = chunk(st + wm * 16 * FM * RA, RA, f, 2 * q4 + h);
    if (!__any((mx_far<FA, FM>(x, w.a) | mx_far<FB, 4>(y, w.b)) != 0)) return false;
    mx_far_products<FA, FB, FM, 4>(x, y, w.a, w.b, acc);
    return true;
  };

#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(kt0 + i, i);
  int slot = 0;
  for (int kt = kt0; kt < kt1; ++kt) {
    wait_vmcnt<LW * (S - 2)>();  // this wave's share of K-tile kt has landed
    barrier_sync();              // everyone's has, and everyone has read K-tile kt - 1
    Words w{};
    if constexpr (EXACT) w = scale_words(smem + opaque_s32(slot * STAGE));
    issue(kt + S - 1, slot == 0 ? S - 1 : slot - 1);
    bool done = false;
    if constexpr (EXACT) done = far_step(slot, w);
    if (!done) compute(slot, w);
    slot = slot + 1 == S ? 0 : slot + 1;
  }
  wait_vmcnt<0>();

  // A lane holds columns 4 r16 .. +3 of rows FM (4 q4 + e) + f.
  const int es = args.out_dtype == 2 ? 4 : 2;
  char* out = args.c + part * args.plane * 4;
  const __amdgpu_buffer_rsrc_t rc = make_rsrc(out + (row0 * args.ldc + col0) * es, ~0ull);
  const int col = 64 * wn + 4 * r16;
  const bool whole = col0 + col + 4 <= args.n;
#pragma unroll
  for (int f = 0; f < FM; ++f)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = 16 * FM * wm + FM * (4 * q4 + e) + f;
      if (row0 + row >= args.m) continue;
      const unsigned off = (unsigned)(row * (int)args.ldc + col) * (unsigned)es;
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = acc[f][j][e];
      if (args.out_dtype == 2) {
        if (whole) {
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]}), rc, off, 0, 0);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (col0 + col + j < args.n) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, v[j]), rc, off + 4 * j, 0, 0);
        }
      } else {
        u32x2 p;
#pragma unroll
        for (int j = 0; j < 2; ++j) p[j] = args.out_dtype == 1 ? pack_bf16(v[2 * j], v[2 * j + 1]) : pack_f16(v[2 * j], v[2 * j + 1]);
        if (whole) {
          __builtin_amdgcn_raw_buffer_store_b64(p, rc, off, 0, 0);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (col0 + col + j < args.n)
              __builtin_amdgcn_raw_buffer_store_b16((unsigned short)(p[j >> 1] >> (16 * (j & 1))), rc, off + 2 * j, 0, 0);
        }
      }
    }
}

template <int FA, int FB, bool EXACT>
static const void* tile_pick(int bm) {
  return bm == 128 ? (const void*)&mx_tile_kernel<FA, FB, EXACT, 4> : bm == 64 ? (const void*)&mx_tile_kernel<FA, FB, EXACT, 2> : (const void*)&mx_tile_kernel<FA, FB, EXACT, 1>;
}
MxEntry mx_tile_entry(int fa, int fb, bool exact, int bm) {
  MxEntry e{nullptr, bm, 128, 256, fa == 4 ? 2 : 1};
  if (fa == 4) e.fn = tile_pick<4, 4, false>(bm);
  else if (fb == 4) e.fn = exact ? tile_pick<8, 4, true>(bm) : tile_pick<8, 4, false>(bm);
  else e.fn = exact ? tile_pick<8, 8, true>(bm) : tile_pick<8, 8, false>(bm);
  return e;
}

}  // namespace spt
