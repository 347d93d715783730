// Products of microscaled operands in 256 x 256 tiles by two wave groups.
//
// Eight waves, two per SIMD, in two groups of four. Between workgroup barriers one group runs the matrix
// instructions of a K-tile while the other reads its fragments from LDS and issues the direct global->LDS loads of a later
// one. A K-tile is 128 bytes of each row: 128 values of 8 bits or 256 of 4 (128 values, 64 bytes, of a 4-bit B beside an
// 8-bit A). Per wave and K-tile that is 32 instructions of 32 cycles or 64 of 16: 1024 cycles either way, and the
// same 24 KiB of LDS reads (16 in the mixed form), the balance of the dense kernel.
//   Group 0 computes rows 0 .. 127 of the tile and group 1 rows 128 .. 255; a group's waves are 2 x 2 of 64 x 128
// outputs, so a group reads its own half of A's tile and both halves of B's. K-tile g is read in phases 2g (group 0) and 2g + 1
// (group 1) and computed in phases 2g + 1 and 2g + 2.
//
// Four rings of half tiles (128 rows, 16 KiB and up to 1 KiB of scales; 153 KiB in all, where whole tiles in five slots fill
// the 160 KiB and leave the scales no room):
//   group 0, phase 2g:     A low (g + 1), 2 slots; B low (g + 1), 2 slots
//   group 1, phase 2g + 1: A high (g + 1), 2 slots; B high (g + 2), 3 slots
// A slot is free again before its load is issued: A halves are read by their own group alone, the phase before last; B low
// (g - 1) was last read in phase 2g - 1, B high (g - 1) as well. Each group waits for its loads at the end of its compute
// phase, a barrier before anyone reads them: A low and B low (g + 1) at the end of phase 2g + 1, A high (g + 1) and B high (g + 2)
// at the end of phase 2g + 2.
//
// The stream of K-tiles runs on across output tiles: a finished tile is stored in its group's next memory phase.
// Rows are staged permuted, so that scales arrive as words and results as 8 neighbouring columns: row r of fragment f is row
// 4r + f of a wave's 64 A rows and 8r + f of its 128 B rows (one word, two words of scales; 16 lanes store 256 or 512
// bytes of a row).
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
  constexpr int LA = 128 * RA / 4096, LB = 128 * RB / 4096, NL = LA + LB + 1;  // loads of a wave in a memory phase
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

  // One operand's stream of K-tiles, at a half tile of 128 rows: descriptors of the half's rows and of the scales that
  // this wave loads (those of 64 rows). Wave-uniform; the tile change stays a branch.
  struct Stream {
    int t, u, kt;
    __amdgpu_buffer_rsrc_t r, s;
  };
  auto set = [&](Stream& st, auto a_c) SPT_INLINE {
    constexpr bool kA = decltype(a_c)::value;
    int tm = 0, tn = 0, part = 0;
    if (st.t < args.units) unit_decode(st.t, args.tiles_m, args.tiles_n, args.group_m, tm, tn, part);
    const int rows = kA ? args.m : args.n, first = (kA ? tm : tn) * 256 + 128 * grp, left = rows - first;
    const int ld = kA ? lda : ldb, block = first / 64 + (v & 1);
    st.kt = part * KT;
    st.r = make_rsrc((kA ? args.a : args.b) + (int64_t)first * ld, left > 0 ? (uint64_t)left * ld : 0);
    st.s = make_rsrc((kA ? args.as : args.bs) + (int64_t)block * sbytes, block * 64 < rows ? (uint64_t)sbytes : 0);
  };
  auto begin = [&](auto a_c) SPT_INLINE {
    Stream st;
    st.t = u0;
    st.u = 0;
    set(st, a_c);
    return st;
  };
  auto advance = [&](Stream& st, auto a_c) SPT_INLINE {
    if (__builtin_expect(++st.u == KT, 0)) {
      st.u = 0;
      st.t += args.grid;
      set(st, a_c);
    }
  };
  using a_ = std::true_type;
  using b_ = std::false_type;

  // This lane's source in a load of 1 KiB: LDS rows 8i .. 8i + 7 (128 bytes) or 16i .. 16i + 15 (64 bytes) of the half.
  const int a_kbyte = ((lane & 7) ^ (lane >> 3)) * 16;
  const unsigned a_off = (unsigned)(4 * (lane >> 3) * lda + a_kbyte);
  const int b_kbyte = (RB == 128 ? (lane & 7) ^ (lane >> 3) : (lane & 3) ^ ((lane >> 3) & 3)) * 16;
  const unsigned b_off = (unsigned)(8 * (RB == 128 ? lane >> 3 : lane >> 2) * ldb + b_kbyte);
  auto a_row = [&](int i) SPT_INLINE { return 64 * (i >> 3) + 32 * (i & 1) + ((i & 7) >> 1); };
  auto b_row = [&](int i) SPT_INLINE { return RB == 128 ? 64 * (i & 1) + (i >> 1) : i; };

  // A memory phase's loads, prepared once and issued one at a time between its reads: A's half at `a`, B's at `b` and the
  // scales of one 64-row block of either, for the slots at LDS offsets `la` and `lb`.
  struct Loads {
    __amdgpu_buffer_rsrc_t ra, rb, rs;
    unsigned va, vb, vs, ka, kb, la, lb, ls;
  };
  auto prepare = [&](const Stream& a, const Stream& b, int la, int lb) SPT_INLINE {
    Loads o;
    const int kta = __builtin_amdgcn_readfirstlane(a.kt + a.u), ktb = __builtin_amdgcn_readfirstlane(b.kt + b.u);
    o.ra = a.r;
    o.rb = b.r;
    o.rs = v < 2 ? a.s : b.s;
    o.ka = (unsigned)(kta * (KS * 16 * FA));
    o.kb = (unsigned)(ktb * (KS * 16 * FB));
    // past the row's end (inside a K-tile of two k-steps, or a part that is shorter than the others), or past the last unit
    o.va = a.t < args.units && (int)o.ka + a_kbyte < lda ? a_off : kOOB;
    o.vb = b.t < args.units && (int)o.kb + b_kbyte < ldb ? b_off : kOOB;
    const int at = (v < 2 ? kta : ktb) * SC + lane * 16;
    o.vs = (v < 2 ? a.t : b.t) < args.units && at < sbytes ? (unsigned)at : kOOB;
    o.la = smem_base + (unsigned)__builtin_amdgcn_readfirstlane(la);
    o.lb = smem_base + (unsigned)__builtin_amdgcn_readfirstlane(lb);
    o.ls = (v < 2 ? o.la + 128 * RA : o.lb + 128 * RB) + (v & 1) * SC;
    return o;
  };
  auto load_one = [&](const Loads& o, auto j_c) SPT_INLINE {
    constexpr int j = decltype(j_c)::value;
    if constexpr (j < LA) {
      const int i = LA * v + j;
      dma16_unseen(o.ra, o.la + i * 1024, add_in_place(o.va, (unsigned)(a_row(i) * lda)), o.ka);
    } else if constexpr (j < LA + LB) {
      const int i = LB * v + j - LA;
      dma16_unseen(o.rb, o.lb + i * 1024, add_in_place(o.vb, (unsigned)(b_row(i) * ldb)), o.kb);
    } else {
      if (lane < 16 * KS) dma16_unseen(o.rs, o.ls, o.vs, 0);
    }
  };
  auto load_all = [&](const Loads& o) SPT_INLINE { static_for<NL>([&](auto j_c) SPT_INLINE { load_one(o, j_c); }); };

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
    const int ua = opaque_s32(__builtin_amdgcn_readfirstlane(a)), ub = opaque_s32(__builtin_amdgcn_readfirstlane(b));
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
    wait_lgkmcnt0();
  };
  // A wave issues its loads at a limited rate: in one burst the reads would queue behind them.
  auto read_with_loads = [&](const Reads& p, const Loads& o) SPT_INLINE {
    static_for<NR>([&](auto i_c) SPT_INLINE {
      constexpr int i = decltype(i_c)::value;
      static_for<NL>([&](auto l_c) SPT_INLINE {
        constexpr int l = decltype(l_c)::value;
        if constexpr (l * NR / NL == i) load_one(o, l_c);
      });
      read_one(p, i_c);
    });
    wait_lgkmcnt0();
  };
  auto compute = [&](auto first_c) SPT_INLINE {
    constexpr bool kFirst = decltype(first_c)::value;
    __builtin_amdgcn_s_setprio(1);
    static_for<KS>([&](auto s_c) SPT_INLINE {
      constexpr int s = decltype(s_c)::value;
      static_for<FM * FN>([&](auto m_c) SPT_INLINE {
        constexpr int m = decltype(m_c)::value, j = m / FM, i = ((j + s) & 1) ? FM - 1 - m % FM : m % FM;
        acc[i][j] = mfma_mx<FA, FB, i, j % 4>(mx_operand<FA>(x[i][s * CA], x[i][s * CA + CA - 1]), mx_operand<FB>(y[j][s * CB], y[j][s * CB + CB - 1]),
                                              (kFirst && s == 0) ? zero : acc[i][j], sx[s], sy[s][j / 4]);
      });
    });
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
  auto a_slot = [&](int p) SPT_INLINE { return (grp ? A_HIGH : A_LOW) + (p & 1) * A_HALF; };
  auto b_low = [&](int p) SPT_INLINE { return B_LOW + (p & 1) * B_HALF; };
  auto b_high = [&](int p3) SPT_INLINE { return B_HIGH + p3 * B_HALF; };
  auto next3 = [&](int p3) SPT_INLINE { return p3 == 2 ? 0 : p3 + 1; };
  int p2 = 0, p3 = 0;  // of the K-tile that is read next

  if (grp == 0) {
    Stream a = begin(a_{}), b = begin(b_{});
    load_all(prepare(a, b, a_slot(0), b_low(0)));
    advance(a, a_{});
    advance(b, b_{});
    wait_vmcnt<0>();
    barrier_sync();
    auto step = [&](auto first_c) SPT_INLINE {
      constexpr bool kFirst = decltype(first_c)::value;
      const Loads o = prepare(a, b, a_slot(p2 + 1), b_low(p2 + 1));
      const Reads r = reads_at(a_slot(p2), wn ? b_high(p3) : b_low(p2));
      if (kFirst && done >= 0) {
        load_all(o);
        epilogue(done);
        read_all(r);
      } else {
        read_with_loads(r, o);
      }
      barrier_sync();
      compute(first_c);
      wait_vmcnt<0>();
      barrier_sync();
      p2 ^= 1;
      p3 = next3(p3);
      advance(a, a_{});
      advance(b, b_{});
    };
    for (int t = u0; units_left > 0; --units_left, t += args.grid) {
      step(std::true_type{});
      for (int u = 1; u < KT; ++u) step(std::false_type{});
      done = t;
    }
    if (done >= 0) epilogue(done);  // beside group 1's last compute phase
    barrier_sync();
  } else {
    Stream a = begin(a_{}), b = begin(b_{});
    load_all(prepare(a, b, a_slot(0), b_high(0)));
    advance(a, a_{});
    advance(b, b_{});
    {  // B high (1); its A half belongs to K-tile 1 too and is loaded again in phase 1
      load_all(prepare(a, b, a_slot(1), b_high(1)));
      advance(b, b_{});
    }
    wait_vmcnt<0>();
    barrier_sync();
    barrier_sync();  // phase 0
    auto step = [&](auto first_c) SPT_INLINE {
      constexpr bool kFirst = decltype(first_c)::value;
      const Loads o = prepare(a, b, a_slot(p2 + 1), b_high(next3(next3(p3))));
      const Reads r = reads_at(a_slot(p2), wn ? b_high(p3) : b_low(p2));
      if (kFirst && done >= 0) {
        load_all(o);
        epilogue(done);
        read_all(r);
      } else {
        read_with_loads(r, o);
      }
      barrier_sync();
      compute(first_c);
      wait_vmcnt<0>();
      barrier_sync();
      p2 ^= 1;
      p3 = next3(p3);
      advance(a, a_{});
      advance(b, b_{});
    };
    for (int t = u0; units_left > 0; --units_left, t += args.grid) {
      step(std::true_type{});
      for (int u = 1; u < KT; ++u) step(std::false_type{});
      done = t;
    }
    if (done >= 0) epilogue(done);
  }
}

template <int FA, int FB>
static const void* pp_pick(int out) {
  return out == 0 ? (const void*)&mx_pp_kernel<FA, FB, 0> : out == 1 ? (const void*)&mx_pp_kernel<FA, FB, 1> : (const void*)&mx_pp_kernel<FA, FB, 2>;
}
MxEntry mx_pp_entry(int fa, int fb, int out) {
  MxEntry e{nullptr, 256, 256, 512, fa == 4 ? 2 : 1, 1};
  e.fn = fa == 4 ? pp_pick<4, 4>(out) : fb == 4 ? pp_pick<8, 4>(out) : pp_pick<8, 8>(out);
  return e;
}

}  // namespace spt
