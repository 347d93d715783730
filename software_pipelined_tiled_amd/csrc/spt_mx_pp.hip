// Products of microscaled operands in 256 x 256 tiles by two wave groups.
//
// Eight waves, two per SIMD, in two groups of four. Between workgroup barriers one group runs the matrix
// instructions of a K-tile while the other reads its fragments from LDS and issues the direct global->LDS loads of a later
// one. A K-tile is 128 bytes of each row: 128 values of 8 bits or 256 of 4 (128 values, 64 bytes, of a 4-bit B beside an
// 8-bit A). Per wave and K-tile that is 32 instructions of 32 cycles or 64 of 16: 1024 cycles either way, and
// 24 KiB of LDS reads (16 in the mixed form), the balance of the dense kernel.
//   Group 0 computes rows 0 .. 127 of the tile and group 1 rows 128 .. 255; a group's waves are 2 x 2 of 64 x 128
// outputs, so a group reads its own half of A's tile and both halves of B's. K-tile g is read in phases 2g (group 0) and 2g + 1
// (group 1) and computed in phases 2g + 1 and 2g + 2.
//
// Four rings of half tiles (128 rows, 16 KiB and up to 1 KiB of scales; 153 KiB in all, where whole tiles in five slots fill
// the 160 KiB and leave the scales no room). Each group loads the half of A that the other computes with, which is free a
// phase earlier:
//   group 0, phase 2g:     B low (g + 1), 2 slots; A high (g + 1), 2 slots
//   group 1, phase 2g + 1: B high (g + 2), 3 slots; A low (g + 2), 2 slots
// A slot's last reader is a barrier ahead of its load: A low (g) is read in phase 2g, A high (g) in 2g + 1, B (g) in both.
// Waits come as late as they may, each with only younger loads still on their way and a barrier before the first reader:
// for B low (g + 1) and the scales at the end of phase 2g + 1 (their loads go out first), for A high (g + 1) at the end of phase
// 2g + 2, for B high and A low (g + 2) at the end of phase 2g + 3. Stores share the count, but loads return in order among
// themselves, so a wait for all but the n youngest loads holds whatever stores lie between.
//
// The stream of K-tiles runs on across output tiles: a finished tile is stored in its group's next memory phase.
// Rows are staged permuted, so that scales arrive as words and results as 8 neighbouring columns: row r of fragment f is row
// 4r + f of a wave's 64 A rows and 8r + f of its 128 B rows (one word, two words of scales; 16 lanes store 256 or 512
// bytes of a row).
//   8192^3, bf16 results: 8 x 8 364 us (3.0 PFLOP/s), 8 x 4 340, 4 x 4 236 (4.7); with 128-row tiles 714, 437 for 8 x 8 and 4 x 4.
// The 8-bit forms keep the matrix cores 0.87 busy (0.82 at 4096 x 8192 x 4096, where a tile has half the k) at 1.5 to 1.55 GHz
// and are held by power. The 4-bit form, 0.60 to 0.64 busy at 1.77 GHz, is held by its memory phases: a K-tile's reads and loads move
// 260 KiB through LDS in the 2048 cycles of its products, which are half as long as the 8-bit ones for as many bytes.
#include "spt_mx_device.h"

namespace spt {

template <int FA, int FB, int OUT>
__global__ void __launch_bounds__(512, 1) mx_pp_kernel(MxGemmArgs args) {
  constexpr int KS = FA == 4 && FB == 4 ? 2 : 1;  // k-steps of a K-tile
  constexpr int RA = 128, RB = FB == 8 || KS == 2 ? 128 : 64;  // bytes of an LDS row
  constexpr int SC = KS * 256;                                 // scale bytes of 64 rows
  constexpr int A_HALF = 128 * RA + 2 * SC, B_HALF = 128 * RB + 2 * SC;
  constexpr int A_LOW = 0, A_HIGH = 2 * A_HALF, B_LOW = 4 * A_HALF, B_HIGH = B_LOW + 2 * B_HALF;
  constexpr int LDS = B_HIGH + 3 * B_HALF;
  constexpr int LA = 128 * RA / 4096, LB = 128 * RB / 4096, NL = LA + LB + KS;  // loads of a wave in a memory phase
  constexpr int FM = 4, FN = 8, CA = FA / 4, CB = FB / 4;                      // fragments; 16-byte chunks of a lane in a k-step
  static_assert(LDS <= 160 * 1024, "the rings fit a compute unit's LDS");
  __shared__ __attribute__((aligned(1024))) char smem[LDS];
  const unsigned smem_base = lds_addr(smem);

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int grp = wave >> 2, v = wave & 3;
  const int wm = v >> 1, wn = v & 1;
  const int r16 = lane & 15, q4 = lane >> 4;
  const int KT = args.per;
  const int lda = args.blocks * (4 * FA), ldb = args.blocks * (4 * FB);
  const int sbytes = args.blocks * kMxScaleRows;  // of 64 rows
  const int u0 = xcd_remap(blockIdx.x, args.grid);

  // This group's stream of K-tiles: descriptors of its half of B's rows, of the other group's half of A's, and of the scales
  // that this wave loads (those of 64 rows: waves 0 and 1 A's, 2 and 3 B's). Wave-uniform; the tile change stays a branch.
  const int kts = (args.ksteps + KS - 1) / KS;
  struct Stream {
    int t, u, kt;
    unsigned past;  // kOOB, past the last unit or past k in a part that is shorter than the others: moves a load out of range
    __amdgpu_buffer_rsrc_t a, b, s;
  };
  auto set = [&](Stream& st) SPT_INLINE {
    int tm = 0, tn = 0, part = 0;
    if (st.t < args.units) unit_decode(st.t, args.tiles_m, args.tiles_n, args.group_m, tm, tn, part);
    const int a0 = tm * 256 + 128 * (1 - grp), b0 = tn * 256 + 128 * grp;
    st.kt = part * KT;
    st.a = make_rsrc(args.a + (int64_t)a0 * lda, a0 < args.m ? (uint64_t)(args.m - a0) * lda : 0);
    st.b = make_rsrc(args.b + (int64_t)b0 * ldb, b0 < args.n ? (uint64_t)(args.n - b0) * ldb : 0);
    const int s0 = (v < 2 ? a0 : b0) + 64 * (v & 1), rows = v < 2 ? args.m : args.n;
    st.s = make_rsrc((v < 2 ? args.as : args.bs) + (int64_t)(s0 / 64) * sbytes, s0 < rows ? (uint64_t)sbytes : 0);
  };
  auto valid = [&](Stream& st) SPT_INLINE { st.past = st.t < args.units && st.kt < kts ? 0u : kOOB; };
  auto enter = [&](Stream& st) SPT_INLINE {  // the next unit, where this one's K-tiles are done
    if (__builtin_expect(st.u == KT, 0)) {
      st.u = 0;
      st.t += args.grid;
      set(st);
    }
  };

  // This lane's source in a load of 1 KiB: LDS rows 8i .. 8i + 7 (128 bytes) or 16i .. 16i + 15 (64 bytes) of the half; the
  // row splits into a part of the lane and one of the instruction.
  const int a_kbyte = ((lane & 7) ^ (lane >> 3)) * 16;
  const unsigned a_off = (unsigned)(4 * (lane >> 3) * lda + a_kbyte);
  const int b_kbyte = (RB == 128 ? (lane & 7) ^ (lane >> 3) : (lane & 3) ^ ((lane >> 3) & 3)) * 16;
  const unsigned b_off = (unsigned)(8 * (RB == 128 ? lane >> 3 : lane >> 2) * ldb + b_kbyte);
  auto a_row = [&](int i) SPT_INLINE { return 64 * (i >> 3) + 32 * (i & 1) + ((i & 7) >> 1); };
  auto b_row = [&](int i) SPT_INLINE { return RB == 128 ? 64 * (i & 1) + (i >> 1) : i; };

  // A memory phase's loads into the slots at LDS offsets la and lb: the scales, B's half, A's half.
  const unsigned s_off = (unsigned)lane * 4;
  struct Loads {
    unsigned va, vb, la, lb, half;
  };
  auto prepare = [&](const Stream& st, int la, int lb) SPT_INLINE {
    Loads o;
    o.va = a_off;
    o.vb = b_off;
    o.half = 0;
    if constexpr (KS == 2) {  // a row may end inside the K-tile; where nothing is loaded anyway (kOOB twice would be 0 again) it does not
      o.half = st.past == 0 && 2 * st.kt + 2 > args.ksteps ? kOOB : 0u;
      o.va = o.half && a_kbyte >= 64 ? kOOB : o.va;
      o.vb = o.half && b_kbyte >= 64 ? kOOB : o.vb;
    }
    o.la = smem_base + (unsigned)la;
    o.lb = smem_base + (unsigned)lb;
    return o;
  };
  auto load_scales = [&](const Stream& st, const Loads& o) SPT_INLINE {
    const unsigned at = (v < 2 ? o.la + 128 * RA : o.lb + 128 * RB) + (v & 1) * SC;
    dma4_unseen(st.s, at, s_off | st.past, (unsigned)(st.kt * SC));
    if constexpr (KS == 2) dma4_unseen(st.s, at + 256, (s_off + 256) | st.past | o.half, (unsigned)(st.kt * SC));
  };
  auto load_one = [&](const Stream& st, const Loads& o, auto j_c) SPT_INLINE {
    constexpr int j = decltype(j_c)::value;
    if constexpr (j < LB) {
      const int i = LB * v + j;
      dma16_unseen(st.b, o.lb + i * 1024, add_in_place(o.vb, (unsigned)(b_row(i) * ldb) | st.past), (unsigned)(st.kt * (KS * 16 * FB)));
    } else {
      const int i = LA * v + j - LB;
      dma16_unseen(st.a, o.la + i * 1024, add_in_place(o.va, (unsigned)(a_row(i) * lda) | st.past), (unsigned)(st.kt * (KS * 16 * FA)));
    }
  };
  auto load_all = [&](const Stream& st, const Loads& o) SPT_INLINE {
    load_scales(st, o);
    static_for<LA + LB>([&](auto j_c) SPT_INLINE { load_one(st, o, j_c); });
  };

  u32x4 x[FM][KS * CA], y[FN][KS * CB];  // the K-tile's fragments: A rows, B rows
  unsigned sx[KS];
  u32x2 sy[KS];
  f32x4 acc[FM][FN];
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};

  // The K-tile's reads in a fixed order. 128-byte rows: lane (r16, q4) takes chunks q4 and 4 + q4 of row r16 of a fragment
  // (in 4 bits one a k-step, in 8 bits both of one).
  const int row_at = r16 * 128, chunk0 = (q4 ^ (r16 & 7)) << 4, chunk1 = ((4 + q4) ^ (r16 & 7)) << 4;
  const int row64_at = r16 * 64 + ((q4 ^ ((r16 >> 1) & 3)) << 4);
  constexpr int NY = FN * KS * CB, NX = FM * KS * CA, NR = NX + NY + 2 * KS;
  struct Reads {
    const char *pa, *pb, *sa, *sb;
  };
  auto reads_at = [&](int a, int b) SPT_INLINE {
    Reads p;
    const int ua = opaque_s32(a), ub = opaque_s32(b);
    p.pa = smem + ua + wm * 64 * RA;
    p.pb = smem + ub;
    p.sa = smem + ua + 128 * RA + wm * SC + q4 * 64 + 4 * r16;
    p.sb = smem + ub + 128 * RB + (r16 >> 3) * SC + q4 * 64 + 8 * (r16 & 7);
    return p;
  };
  auto read_one = [&](const Reads& p, auto i_c) SPT_INLINE {
    constexpr int i = decltype(i_c)::value;
    if constexpr (i < 2 * KS) {
      constexpr int s = i / 2;
      if constexpr (i % 2 == 0) sx[s] = *(const unsigned*)(p.sa + s * 256);
      else sy[s] = *(const u32x2*)(p.sb + s * 256);
    } else if constexpr (i < 2 * KS + NY) {
      constexpr int f = (i - 2 * KS) / (KS * CB), c = (i - 2 * KS) % (KS * CB);
      if constexpr (RB == 128) y[f][c] = *(const u32x4*)(p.pb + f * 16 * 128 + row_at + (c ? chunk1 : chunk0));
      else y[f][c] = *(const u32x4*)(p.pb + f * 16 * 64 + row64_at);
    } else {
      constexpr int f = (i - 2 * KS - NY) / (KS * CA), c = (i - 2 * KS - NY) % (KS * CA);
      x[f][c] = *(const u32x4*)(p.pa + f * 16 * 128 + row_at + (c ? chunk1 : chunk0));
    }
  };
  auto read_all = [&](const Reads& p) SPT_INLINE {
    static_for<NR>([&](auto i_c) SPT_INLINE { read_one(p, i_c); });
  };
  // A wave issues its loads at a limited rate (1 KiB in about 56 cycles): in one burst the reads would queue behind them.
  // Among the matrix instructions they hold those up as long (8192^3 8 x 8: 405 us).
  auto read_with_loads = [&](const Reads& p, const Stream& st, const Loads& o) SPT_INLINE {
    load_scales(st, o);
    static_for<NR>([&](auto i_c) SPT_INLINE {
      constexpr int i = decltype(i_c)::value;
      static_for<LA + LB>([&](auto l_c) SPT_INLINE {
        constexpr int l = decltype(l_c)::value;
        if constexpr (l * NR / (LA + LB) == i) load_one(st, o, l_c);
      });
      read_one(p, i_c);
    });
  };
  // The products of the K-tile in registers, and nothing else: scalar instructions between them, a few at a time, made this phase
  // 1013 -> 1250 cycles.
  auto compute = [&](auto first_c) SPT_INLINE {
    constexpr bool kFirst = decltype(first_c)::value;
    __builtin_amdgcn_s_setprio(1);
    static_for<KS * FM * FN>([&](auto m_c) SPT_INLINE {
      constexpr int m = decltype(m_c)::value, s = m / (FM * FN), j = m % (FM * FN) / FM, i = ((j + s) & 1) ? FM - 1 - m % FM : m % FM;
      acc[i][j] = mfma_mx<FA, FB, i, j % 4>(mx_operand<FA>(x[i][s * CA], x[i][s * CA + CA - 1]), mx_operand<FB>(y[j][s * CB], y[j][s * CB + CB - 1]),
                                            (kFirst && s == 0) ? zero : acc[i][j], sx[s], sy[s][j / 4]);
    });
    // The products belong here: without a use the compiler sinks them past the barrier to the sums' next use, in front of the
    // group's own reads (8192^3 8 x 8: 455 us, 362 with it).
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        f32x4& c = acc[i][j];
        asm volatile("" : "+v"(c));
      }
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(0);
  };

  // This wave's part of unit t from the accumulators: for each (f, e) 8 columns of row 16 q4 + 4e + f.
  constexpr int es = OUT == 2 ? 4 : 2;
  auto epilogue = [&](int t) SPT_INLINE {
    int tm, tn, part;
    unit_decode(__builtin_amdgcn_readfirstlane(t), args.tiles_m, args.tiles_n, args.group_m, tm, tn, part);
    const int row0 = tm * 256, col0 = tn * 256, ldc = (int)args.ldc;
    const __amdgpu_buffer_rsrc_t rc = make_rsrc(args.c + part * args.plane * 4 + (int64_t)row0 * args.ldc * es,
                                                ((uint64_t)(args.m - row0 - 1) * args.ldc + args.n) * es);
    const int ln = (int)opaque_u32((unsigned)lane);
    const int m_lane = 128 * grp + 64 * wm + 16 * (ln >> 4), n_lane = col0 + 128 * wn + 8 * (ln & 15);
    const unsigned voff = (unsigned)(m_lane * ldc + n_lane) * (unsigned)es;
    const bool full = args.m - row0 >= 256 && args.n - col0 >= 256;
    auto stores = [&](auto mode_c) SPT_INLINE {
      constexpr int kMode = decltype(mode_c)::value;
      static_for<16>([&](auto st_c) SPT_INLINE {
        constexpr int f = decltype(st_c)::value % 4, e = decltype(st_c)::value / 4;
        float vv[8];
#pragma unroll
        for (int j = 0; j < FN; ++j) vv[j] = acc[f][j][e];
        if constexpr (kMode == 0) store8_at<OUT, kStoreNonTemporal>(vv, rc, voff, (unsigned)((4 * e + f) * ldc * es));
        else if constexpr (kMode == 1) store8_at<OUT>(vv, rc, voff, (unsigned)((4 * e + f) * ldc * es));
        else store8<OUT, true>(vv, rc, m_lane + 4 * e + f, args.m - row0, n_lane, args.n, ldc);
        __builtin_amdgcn_sched_barrier(0);
      });
    };
    if (full && args.nt) stores(std::integral_constant<int, 0>{});
    else if (full) stores(std::integral_constant<int, 1>{});
    else stores(std::integral_constant<int, 2>{});
  };

  int units_left = u0 < args.units ? (args.units - u0 - 1) / args.grid + 1 : 0;
  int done = -1;  // the unit whose stores are pending
  // Ring positions of K-tile g: parity for the rings of two, g mod 3 for B high.
  auto a_low = [&](int p) SPT_INLINE { return A_LOW + (p & 1) * A_HALF; };
  auto a_high = [&](int p) SPT_INLINE { return A_HIGH + (p & 1) * A_HALF; };
  auto b_low = [&](int p) SPT_INLINE { return B_LOW + (p & 1) * B_HALF; };
  auto b_high = [&](int p3) SPT_INLINE { return B_HIGH + p3 * B_HALF; };
  auto next3 = [&](int p3) SPT_INLINE { return p3 == 2 ? 0 : p3 + 1; };
  Stream st;
  st.t = u0;
  st.u = 0;
  set(st);
  valid(st);
  // What the next memory phase does: the slots of the K-tile it reads, and those of its loads.
  int p2 = 0, p3 = 0, ra = 0, rb = 0, la = 0, lb = 0;
  auto plan = [&]() SPT_INLINE {
    ra = opaque_s32(grp ? a_high(p2) : a_low(p2));
    rb = opaque_s32(wn ? b_high(p3) : b_low(p2));
    la = opaque_s32(grp ? a_low(p2) : a_high(p2 + 1));
    lb = opaque_s32(grp ? b_high(next3(next3(p3))) : b_low(p2 + 1));
  };
  // A group's memory phase and compute phase of one K-tile. A finished tile's stores go out between the loads and the reads.
  // The next memory phase's scalar work is done while the reads are on their way.
  auto step = [&](auto first_c, auto group0_c) SPT_INLINE {
    const Loads o = prepare(st, la, lb);
    const Reads r = reads_at(ra, rb);
    const bool stores = decltype(first_c)::value && done >= 0;
    if (stores) {
      load_all(st, o);
      wait_vmcnt<NL>();  // this group's loads of its last memory phase have landed
      epilogue(done);
      read_all(r);
    } else {
      read_with_loads(r, st, o);
    }
    ++st.u;
    ++st.kt;
    enter(st);
    valid(st);
    p2 ^= 1;
    p3 = next3(p3);
    plan();
    wait_lgkmcnt0();
    if (!stores) wait_vmcnt<NL>();
    barrier_sync();
    compute(first_c);
    if constexpr (decltype(group0_c)::value) wait_vmcnt<LA>();  // the scales and B low have landed
    barrier_sync();
  };
  auto run = [&](auto group0_c) SPT_INLINE {
    for (int t = u0; units_left > 0; --units_left, t += args.grid) {
      step(std::true_type{}, group0_c);
      for (int u = 1; u < KT; ++u) step(std::false_type{}, group0_c);
      done = t;
    }
    if (done >= 0) epilogue(done);  // group 0's beside group 1's last compute phase
  };

  auto first_loads = [&](int a, int b) SPT_INLINE {
    load_all(st, prepare(st, a, b));
    ++st.u;
    ++st.kt;
    enter(st);
    valid(st);
  };
  if (grp == 0) {
    first_loads(a_high(0), b_low(0));
    wait_vmcnt<0>();
    barrier_sync();
    plan();
    run(std::true_type{});
    barrier_sync();
  } else {
    first_loads(a_low(0), b_high(0));
    first_loads(a_low(1), b_high(1));
    wait_vmcnt<0>();
    barrier_sync();
    barrier_sync();  // phase 0
    plan();
    run(std::false_type{});
  }
  wait_vmcnt<0>();  // no load to LDS outlives the workgroup
}

template <int FA, int FB>
static const void* pp_pick(int out) {
  return out == 0 ? (const void*)&mx_pp_kernel<FA, FB, 0> : out == 1 ? (const void*)&mx_pp_kernel<FA, FB, 1> : (const void*)&mx_pp_kernel<FA, FB, 2>;
}
MxEntry mx_pp_entry(int fa, int fb, int out) {
  MxEntry e{nullptr, 256, 256, 512, fa == 4 ? 2 : 1};
  e.fn = fa == 4 ? pp_pick<4, 4>(out) : fb == 4 ? pp_pick<8, 4>(out) : pp_pick<8, 8>(out);
  return e;
}

}  // namespace spt
