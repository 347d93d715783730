// The experts' products in 256 x 256 tiles by two wave groups: the phase stream of the dense two-group
// kernel (spt_gemm_pp.hip) over units of work that differ in their expert, their operands' bases and
// their number of K-tiles.
//
// Eight waves, two per SIMD, in two groups of four. Between workgroup barriers one group runs the
// matrix instructions of a K-tile (64 deep) while the other reads its fragments from LDS and issues the
// direct global->LDS loads of a later one. K-tile g is read in phases 2g (group 0) and 2g+1 (group 1) and
// computed in phases 2g+1 and 2g+2. Five 32 KiB operand slots: K-tile g's X tile sits in slot 2g mod 5 and
// its Y tile in slot 2g+1 mod 5; group 0 loads Y(g+1) in phase 2g, group 1 X(g+2) in phase 2g+1. The
// stream runs on across units: a unit's stores go out in its group's next memory phase. A unit without a
// sum (an expert without rows in grad B; rows that belong to no expert) is one K-tile of zeros.
//
// What differs by mode is the side on which an operand is contiguous (spt_grouped.hip):
//   * contiguous in c: 256 rows of 64 c, as in the dense kernel;
//   * contiguous in i or j: 64 rows of c by 256 columns, 512 bytes a row, turned by the transposing LDS
//     read (spt_transpose.h). Its loads' descriptor starts at the K-tile's first row and ends at the
//     expert's last, so rows past it read zeros.
// Forward keeps the dense kernel's fragment order (a lane holds 8 consecutive columns of four rows). A
// transposing read gives a quarter-wave 16 columns as they lie, so the gradients feed Y as the matrix
// instruction's first operand: a lane then holds four consecutive columns of one row per fragment, and an
// exchange between quarter-waves makes them eight per fragment pair.
//
// What bounds it: the matrix cores at the clock the power limit allows. 16384 rows, 8 experts of 8192 x 4096, bf16:
// forward 779 to 811 us in a loop, 1356 to 1411 TFLOP/s (838 the median of a trace), the matrix cores 0.84 busy (grad
// A 0.79, grad B 0.65, since its sums of 2048 rows end in stores twice as often); the dense kernel of this library
// reaches 1488 TFLOP/s at 8192^3. No read of LDS has
// a bank conflict. What is left: the last round of tiles, which is as long as a full one (328 tiles over 256
// compute units: 189 us where 256 take 100), and grad B's fp32 stores (8190 rows, 16 experts of 4096 x 2048: 218 us with its
// operands in the caches, 132 without the stores), which go out while one of the two groups computes and take longer
// than that. In a training step, where operands come from HBM, it takes 234 us with even experts and 261 to 291 with
// uneven ones: a workgroup's tiles are every 256th, whatever their sums' lengths.
#include "spt_device.h"
#include "spt_experts.h"
#include "spt_transpose.h"

namespace spt {

struct PpUnit {
  int t;   // unit number; -1: past the last
  int e, row0, col0, rows_left, cols_left;
  int c0, kc, kt;  // first row of the sum (grad B), its length, its K-tiles
};

template <int MODE, typename TIn, int OUT>
__global__ void __launch_bounds__(512, 1) grouped_pp_kernel(GroupedArgs args) {
  constexpr bool TX = MODE == kGroupedGradB, TY = MODE != kGroupedForward;
  constexpr int BM = 256, BN = 256, BK = 64, S = 5;
  constexpr int TM = 64, TN = 128;
  constexpr int FM = TM / 16, FN = TN / 16, NSUB = 2;
  constexpr int SLOT = BM * BK * 2;
  constexpr PipeProtocol P = pipe_protocol(BM, BN, BK, S, 8);
  constexpr int LA = P.la;  // loads per wave for one operand tile
  static_assert(LA == SLOT / 1024 / 4 && P.lb == LA && S * SLOT <= 160 * 1024, "one group of four waves loads a tile");
  __shared__ __attribute__((aligned(1024))) char smem[S * SLOT];
  const unsigned smem_base = lds_addr(smem);

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int grp = wave >> 2, v = wave & 3;
  const int wm = v >> 1, wn = v & 1;
  constexpr int es = OUT == 2 ? 4 : 2;
  const int m_base = 128 * grp + TM * wm;
  const int ldx = (int)args.ldx, ldy = (int)args.ldy, ldc = (int)args.ldc;

  // unit t: its expert, output tile and sum
  auto unit_at = [&](int t) SPT_INLINE {
    PpUnit u;
    int tm = 0, tn = 0;
    u.t = -1;
    u.e = u.row0 = u.col0 = u.rows_left = u.cols_left = u.c0 = u.kc = 0;
    if constexpr (MODE == kGroupedGradB) {
      const int per = args.tiles_m * args.tiles_n;
      if (t < args.units) {
        u.t = t;
        u.e = t / per;
        grouped_raster(t - u.e * per, args.tiles_m, args.tiles_n, args.group_m, tm, tn);
        u.row0 = tm * BM;
        u.rows_left = args.m - u.row0;
        u.c0 = clampi(args.offsets[u.e], 0, args.rows);
        u.kc = clampi(args.offsets[u.e + 1], u.c0, args.rows) - u.c0;
        u.c0 = __builtin_amdgcn_readfirstlane(u.c0);
        u.kc = __builtin_amdgcn_readfirstlane(u.kc);
      }
    } else if (t < args.units) {
      const GroupBlock g = find_group(args.offsets, args.experts, args.rows, BM, args.tiles_n, args.rest != 0, t);
      if (g.e >= 0) {
        u.t = t;
        u.e = g.e;
        grouped_raster(g.local, g.blocks, args.tiles_n, args.group_m, tm, tn);
        u.row0 = g.begin + tm * BM;
        u.rows_left = g.end - u.row0;
        u.kc = g.e == args.experts ? 0 : args.kc;
      }
    }
    u.col0 = tn * BN;
    u.cols_left = args.n - u.col0;
    u.kt = u.kc > BK ? (u.kc + BK - 1) / BK : 1;
    return u;
  };

  // ------------------------------------------------------------------------ loads
  // Wave v's load j of an operand tile fills LDS bytes [1024 (LA v + j), +1024). Contiguous in c: rows
  // 8q .. 8q+7 (q = LA v + j), lane l row 8q + l/8, physical chunk l%8. Else: c rows 2q, 2q+1, lane l row
  // 2q + l/32, physical chunk l%32, logical chunk (l%32) XOR 2 tr_swz(c). With LA = 8 the XOR is the lane's
  // part l/32 and the load's: 32 columns for an odd j, 64 for j of 4 and more.
  const int lrow = lane >> 3, lane_kc = 8 * ((lane & 7) ^ swz(lrow));
  const int trow = lane >> 5, tcol = 8 * ((lane & 31) ^ (2 * trow));
  static_assert(LA == 8, "the swizzle's split into lane and load");
  struct Cursor {
    PpUnit tl;
    int u;
    __amdgpu_buffer_rsrc_t rx, ry;  // operands contiguous in c: the whole sum
    const char *xb, *yb;            // others: the unit's first c row
  };
  auto set_bases = [&](Cursor& c) SPT_INLINE {
    const int kc8 = (c.tl.kc + 7) & ~7;  // memory rows hold a multiple of 8 elements, zeros past kc
    if constexpr (TX) c.xb = args.X + ((int64_t)c.tl.c0 * args.ldx + c.tl.row0) * 2;
    else c.rx = make_rsrc(args.X + (int64_t)c.tl.row0 * args.ldx * 2, ((uint64_t)(c.tl.rows_left - 1) * args.ldx + kc8) * 2);
    if constexpr (MODE == kGroupedGradB) c.yb = args.Y + ((int64_t)c.tl.c0 * args.ldy + c.tl.col0) * 2;
    else if constexpr (MODE == kGroupedGradA) c.yb = args.Y + ((int64_t)c.tl.e * args.sy + c.tl.col0) * 2;
    else c.ry = make_rsrc(args.Y + ((int64_t)c.tl.e * args.sy + (int64_t)c.tl.col0 * args.ldy) * 2,
                          ((uint64_t)(c.tl.cols_left - 1) * args.ldy + kc8) * 2);
  };
  auto advance = [&](Cursor& c) SPT_INLINE {
    if (c.tl.t >= 0 && __builtin_expect(++c.u == c.tl.kt, 0)) {
      c.u = 0;
      c.tl = unit_at(c.tl.t + args.grid);
      set_bases(c);
    }
  };
  auto cursor_at = [&](const PpUnit& u) SPT_INLINE {
    Cursor c;
    c.tl = u;
    c.u = 0;
    set_bases(c);
    return c;
  };
  auto valid = [&](const Cursor& c) SPT_INLINE { return c.tl.t >= 0; };

  // Y's row in LDS row r, where Y is contiguous in c. 16-bit outputs: b_row_perm128. fp32 outputs: in each 64
  // rows, LDS row 16 f + c holds row 4 c + f, so that a lane holds four consecutive columns per four
  // fragments, 16 bytes, and a quarter-wave 256.
  auto y_row = [](int r) SPT_INLINE {
    return OUT == 2 ? (r & ~63) + 4 * (r & 15) + ((r >> 4) & 3) : b_row_perm128(r);
  };
  struct OpLoads {
    __amdgpu_buffer_rsrc_t r;
    unsigned v0, lds, soff;  // v0: the lane's offset; contiguous in i or j: of its row alone
    int ld;
  };
  // the descriptor of a K-tile's c rows (operand contiguous in i or j): from its first to the sum's last
  auto rows_rsrc = [&](const Cursor& c, const char* base, int64_t ld, int left) SPT_INLINE {
    const int k0 = __builtin_amdgcn_readfirstlane(c.u) * BK;
    const int rows = __builtin_amdgcn_readfirstlane(c.tl.kc) - k0;
    const int64_t bytes = rows > 0 ? ((rows - 1) * ld + ((left + 7) & ~7)) * 2 : 0;
    return make_rsrc(base + (int64_t)k0 * ld * 2, (uint64_t)bytes);
  };
  auto prep = [&](const Cursor& c, bool x, int dst) SPT_INLINE {
    OpLoads o;
    const int k0 = __builtin_amdgcn_readfirstlane(c.u) * BK;
    o.lds = smem_base + (unsigned)__builtin_amdgcn_readfirstlane(dst) + LA * v * 1024;
    o.ld = x ? ldx : ldy;
    if (x ? TX : TY) {
      o.r = x ? rows_rsrc(c, c.xb, args.ldx, c.tl.rows_left) : rows_rsrc(c, c.yb, args.ldy, c.tl.cols_left);
      o.v0 = (unsigned)(trow * o.ld) * 2u;
      o.soff = 0;
    } else {
      o.r = x ? c.rx : c.ry;
      const int row = x ? lrow : y_row(lrow);
      o.v0 = lane_kc < c.tl.kc - k0 ? (unsigned)(row * o.ld + lane_kc) * 2u : kOOB;
      o.soff = 2u * k0;
    }
    return o;
  };
  auto load_one = [&](const OpLoads& o, bool x, int j) SPT_INLINE {
    const int q = LA * v + j;
    if (x ? TX : TY) {
      // the row rides in the scalar offset, which the descriptor's end counts too
      dma16_unseen(o.r, o.lds + j * 1024, xor_add_in_place(2u * tcol, 64u * (j & 1) + 128u * (j >> 2), o.v0),
                   (unsigned)(2 * q * o.ld) * 2u);
    } else {
      const int row = x ? 8 * q : y_row(8 * q);
      dma16_unseen(o.r, o.lds + j * 1024, add_in_place(o.v0, (unsigned)(row * o.ld) * 2u), o.soff);
    }
  };
  auto issue = [&](const Cursor& c, bool x, int dst) SPT_INLINE {
    const OpLoads o = prep(c, x, dst);
#pragma unroll
    for (int j = 0; j < LA; ++j) load_one(o, x, j);
  };
  auto x_at = [&](int p) SPT_INLINE { return p * SLOT; };
  auto y_at = [&](int p) SPT_INLINE { return (p + 1 == S ? 0 : p + 1) * SLOT; };
  auto pos_step = [&](int p, int n) SPT_INLINE {
    const int q = p + 2 * n;
    return q >= S ? q - S : q;
  };

  // ------------------------------------------------------------------------ fragments
  u32x4 yf[NSUB][FN], xf[NSUB][FM];
  f32x4 acc[FN][FM];
  const f32x4 zero4 = {0.f, 0.f, 0.f, 0.f};

  // LDS byte offsets of the lane's reads. Contiguous in c: one per k-step, fragments 16 rows apart. Else:
  // the lane's c row is 32 s + 8 (l/16) + 4 u + (l%16)/4 (s, u as immediates), so the swizzle is the lane's
  // own, and fragment f's 32 bytes are its first fragment's XOR 32 f.
  const int p16 = lane & 15, h16 = lane >> 4;
  int x_rd[TX ? 1 : NSUB], y_rd[TY ? 1 : NSUB];
  if constexpr (TX) {
    x_rd[0] = tr_offset<BM>(8 * h16 + (p16 >> 2), m_base / 16) + 8 * (p16 & 3);
  } else {
#pragma unroll
    for (int s = 0; s < NSUB; ++s) x_rd[s] = lds_chunk_offset(BM, m_base + p16, 4 * s + h16);
  }
  if constexpr (TY) {
    y_rd[0] = tr_offset<BN>(8 * h16 + (p16 >> 2), TN * wn / 16) + 8 * (p16 & 3);
  } else {
#pragma unroll
    for (int s = 0; s < NSUB; ++s) y_rd[s] = lds_chunk_offset(BN, TN * wn + p16, 4 * s + h16);
  }
  unsigned x_addr = 0, y_addr = 0;
  constexpr int NR = NSUB * (FN + FM);
  // Slots are multiples of 32 KiB and the array is the kernel's only LDS, so a slot's offset, a fragment's
  // 32 f and the lane's offset meet in one XOR.
  struct Bases {
    const char *px, *py;
    unsigned sx, sy;
  };
  auto frag_bases = [&](int p) SPT_INLINE {
    const int pu = __builtin_amdgcn_readfirstlane(p);
    Bases b;
    const int x = opaque_s32(x_at(pu)), y = opaque_s32(y_at(pu));
    b.px = smem + x;
    b.py = smem + y;
    b.sx = smem_base ^ (unsigned)x;
    b.sy = smem_base ^ (unsigned)y;
    return b;
  };
  // Read i of NR: Y's fragments, then X's. A transposed operand's two k-steps of a fragment follow each
  // other, since they share an address register.
  auto read_one = [&](auto i_c, const Bases& b) SPT_INLINE {
    constexpr int i = decltype(i_c)::value;
    if constexpr (i < NSUB * FN) {
      constexpr int s = TY ? i % NSUB : i / FN, f = TY ? i / NSUB : i % FN;
      if constexpr (TY) {
        if constexpr (s == 0) y_addr = xor_in_place((unsigned)y_rd[0], b.sy ^ (32u * f));
        yf[s][f] = tr_frag<2 * BN>((lds_void_t*)(uintptr_t)(y_addr + s * (64 * BN)));
      } else {
        yf[s][f] = *(const u32x4*)(b.py + y_rd[s] + f * 2048);
      }
    } else {
      constexpr int i2 = i - NSUB * FN, s = TX ? i2 % NSUB : i2 / FM, j = TX ? i2 / NSUB : i2 % FM;
      if constexpr (TX) {
        if constexpr (s == 0) x_addr = xor_in_place((unsigned)x_rd[0], b.sx ^ (32u * j));
        xf[s][j] = tr_frag<2 * BM>((lds_void_t*)(uintptr_t)(x_addr + s * (64 * BM)));
      } else {
        xf[s][j] = *(const u32x4*)(b.px + x_rd[s] + j * 2048);
      }
    }
  };
  auto read_frags = [&](int p) SPT_INLINE {
    const Bases b = frag_bases(p);
    static_for<NR>([&](auto i_c) { read_one(i_c, b); });
    wait_lgkmcnt0();
  };
  // the reads with the operand's LA loads spread between them
  auto read_frags_with_loads = [&](int p, auto&& load) SPT_INLINE {
    const Bases b = frag_bases(p);
    static_for<NR>([&](auto i_c) {
      constexpr int i = decltype(i_c)::value;
      static_for<LA>([&](auto l_c) {
        constexpr int l = decltype(l_c)::value;
        if constexpr (l * NR / LA == i) load(l);
      });
      read_one(i_c, b);
    });
    wait_lgkmcnt0();
  };
  auto compute = [&](auto first_c) SPT_INLINE {
    constexpr bool kFirst = decltype(first_c)::value;
    __builtin_amdgcn_s_setprio(1);
    static_for<NSUB>([&](auto s_c) {
      constexpr int s = decltype(s_c)::value;
      static_for<FN * FM>([&](auto m_c) {
        constexpr int m = decltype(m_c)::value, i = m / FM, j = ((i + s) & 1) ? FM - 1 - m % FM : m % FM;
        const f32x4 c = (kFirst && s == 0) ? zero4 : acc[i][j];
        if constexpr (TY) acc[i][j] = mfma16<TIn>(yf[s][i], xf[s][j], c);
        else acc[i][j] = mfma16<TIn>(xf[s][j], yf[s][i], c);
      });
    });
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(0);
  };

  // ------------------------------------------------------------------------ stores
  // 16-bit outputs, 16 stores of eight columns. Forward: store s is row 4 (l/16) + s%4 of X block s/4, columns
  // 8 (l%16) .. +7. Gradients: row l%16 of X block s/4, Y block pair s%4. fp32 outputs, 32 stores of four
  // columns: half s%2 of a row (forward), or Y block s%8 (gradients). The stores that fill one 128-byte line
  // follow each other: four apart, grad B ran 5 % (16-bit) and 12 % (fp32) slower.
  auto epilogue = [&](const PpUnit& in, auto reads_c, int p) SPT_INLINE {
    constexpr bool kReads = decltype(reads_c)::value;
    const int e = __builtin_amdgcn_readfirstlane(in.e), row0 = __builtin_amdgcn_readfirstlane(in.row0);
    const int col0 = __builtin_amdgcn_readfirstlane(in.col0), rows_left = __builtin_amdgcn_readfirstlane(in.rows_left);
    const int cols_left = __builtin_amdgcn_readfirstlane(in.cols_left);
    const __amdgpu_buffer_rsrc_t rc =
        make_rsrc(args.C + ((MODE == kGroupedGradB ? (int64_t)e * args.sc : 0) + (int64_t)row0 * args.ldc) * es,
                  ((uint64_t)(rows_left - 1) * args.ldc + args.n) * es);
    const int ln = (int)opaque_u32((unsigned)lane);
    const int m_lane = TY ? m_base + ln % 16 : m_base + 4 * (ln / 16);
    const int n_lane = col0 + TN * wn + (OUT == 2 ? 4 * (TY ? ln / 16 : ln % 16) : TY ? pair_column(ln) : 8 * (ln % 16));
    const unsigned voff = (unsigned)(m_lane * ldc + n_lane) * (unsigned)es;
    // 0: interior, non-temporal; 1: interior, default policy; 2: edge tile, masked per element
    auto stores = [&](auto mode_c) SPT_INLINE {
      constexpr bool kEdge = decltype(mode_c)::value == 2;
      constexpr int kPolicy = decltype(mode_c)::value == 0 ? kStoreNonTemporal : 0;
      Bases b{};
      if constexpr (kReads) b = frag_bases(p);
      constexpr int NS = OUT == 2 ? 32 : 16;
      static_for<NS>([&](auto s_c) {
        constexpr int st = decltype(s_c)::value;
        if constexpr (OUT == 2) {
          constexpr int j = st / 8, e = st / 2 % 4, half = st % 2;  // e, half: forward
          constexpr int dm = TY ? 16 * j : 16 * j + e, dn = TY ? 16 * (st % 8) : 64 * half;
          f32x4 v;
          if constexpr (TY) v = acc[st % 8][j];
          else {
#pragma unroll
            for (int f = 0; f < 4; ++f) v[f] = acc[4 * half + f][j][e];
          }
          if constexpr (kEdge) store4_f32<true>(v, rc, m_lane + dm, rows_left, n_lane + dn, args.n, ldc);
          else __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rc, voff, (unsigned)((dm * ldc + dn) * es), kPolicy);
        } else {
          constexpr int dm = TY ? 16 * (st / 4) : 16 * (st / 4) + st % 4, dn = TY ? 32 * (st % 4) : 0;
          float vv[8];
          if constexpr (TY) {
            pair_columns(acc[2 * (st % 4)][st / 4], acc[2 * (st % 4) + 1][st / 4], vv);
          } else {
#pragma unroll
            for (int f = 0; f < 8; ++f) vv[f] = acc[f][st / 4][st % 4];
          }
          if constexpr (kEdge) store8<OUT, true>(vv, rc, m_lane + dm, rows_left, n_lane + dn, args.n, ldc);
          else store8_at<OUT, kPolicy>(vv, rc, voff, (unsigned)((dm * ldc + dn) * es));
        }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (kReads) {
          static_for<NR>([&](auto r_c) {
            if constexpr (decltype(r_c)::value * NS / NR == st) read_one(r_c, b);
          });
        }
      });
      if constexpr (kReads) wait_lgkmcnt0();
    };
    if (rows_left < BM || cols_left < BN) stores(std::integral_constant<int, 2>{});
    else if (!TY || args.nt) stores(std::integral_constant<int, 0>{});
    else stores(std::integral_constant<int, 1>{});
  };
  using t_ = std::true_type;
  using f_ = std::false_type;
  // the previous unit's stores (if any), then K-tile g's fragments; the reads go out between the stores
  // where the registers allow it (forward, 16-bit outputs)
  auto store_and_read = [&](const PpUnit& prev, int p) SPT_INLINE {
    if (prev.t >= 0) {
      if constexpr (OUT == 2 || TY) {
        epilogue(prev, f_{}, 0);
        read_frags(p);
      } else {
        epilogue(prev, t_{}, p);
      }
    } else {
      read_frags(p);
    }
  };

  PpUnit cur = unit_at(xcd_remap(blockIdx.x, args.grid));
  if (cur.t < 0) return;  // every wave takes this branch: no barrier is left waiting
  PpUnit prev;
  prev.t = -1;
  int p = 0;
  if (grp == 0) {
    Cursor c0 = cursor_at(cur), nx = c0;  // nx: K-tile g+1
    advance(nx);
    issue(c0, true, x_at(0));
    issue(c0, false, y_at(0));
    if (valid(nx)) {
      issue(nx, true, x_at(pos_step(0, 1)));
      wait_vmcnt<P.pp_g0_prologue_wait>();  // K-tile 0 landed; X(1) may be in flight
    } else {
      wait_vmcnt<0>();
    }
    barrier_sync();
    auto step = [&](auto first_c) SPT_INLINE {
      // phase 2g: load Y(g+1), store the previous unit, read K-tile g
      if constexpr (decltype(first_c)::value) {
        if (valid(nx)) issue(nx, false, y_at(pos_step(p, 1)));
        store_and_read(prev, p);
      } else {
        if (valid(nx)) {
          const OpLoads o = prep(nx, false, y_at(pos_step(p, 1)));
          read_frags_with_loads(p, [&](int j) SPT_INLINE { load_one(o, false, j); });
        } else {
          read_frags(p);
        }
      }
      barrier_sync();
      // phase 2g+1: compute, then wait for this group's loads of K-tile g+1 and its stores
      compute(first_c);
      wait_vmcnt<0>();
      barrier_sync();
      p = pos_step(p, 1);
      advance(nx);
    };
    for (; cur.t >= 0; cur = unit_at(cur.t + args.grid)) {
      step(t_{});
      for (int u = 1; u < cur.kt; ++u) step(f_{});
      prev = cur;
    }
    epilogue(prev, f_{}, 0);  // phase 2G, beside group 1's last matrix instructions
    barrier_sync();
  } else {
    Cursor n2 = cursor_at(cur);  // K-tile g+2
    advance(n2);
    advance(n2);
    barrier_sync();  // K-tile 0 visible
    barrier_sync();  // phase 0: idle
    auto step = [&](auto first_c) SPT_INLINE {
      constexpr bool kFirst = decltype(first_c)::value;
      // phase 2g+1: load X(g+2), read K-tile g, make sure X(g+1) has landed. In a unit's first K-tile
      // the wait comes before the previous unit's stores, so that it counts loads only.
      bool loaded = false;
      auto wait_x = [&]() SPT_INLINE {
        if (loaded) wait_vmcnt<P.pp_g1_wait>();
        else wait_vmcnt<0>();
      };
      if constexpr (kFirst) {
        if (valid(n2)) {
          issue(n2, true, x_at(pos_step(p, 2)));
          loaded = true;
        }
        wait_x();
        store_and_read(prev, p);
      } else {
        if (valid(n2)) {
          const OpLoads o = prep(n2, true, x_at(pos_step(p, 2)));
          read_frags_with_loads(p, [&](int j) SPT_INLINE { load_one(o, true, j); });
          loaded = true;
        } else {
          read_frags(p);
        }
        wait_x();
      }
      barrier_sync();
      compute(first_c);  // phase 2g+2
      barrier_sync();
      p = pos_step(p, 1);
      advance(n2);
    };
    for (; cur.t >= 0; cur = unit_at(cur.t + args.grid)) {
      step(t_{});
      for (int u = 1; u < cur.kt; ++u) step(f_{});
      prev = cur;
    }
    epilogue(prev, f_{}, 0);
  }
}

template <int MODE>
static const void* pp_pick(int bf16, int out) {
#define SPT_GROUPED_PP(TI, O) (const void*)&grouped_pp_kernel<MODE, TI, O>
  static const void* const fn[2][3] = {
      {SPT_GROUPED_PP(_Float16, 0), SPT_GROUPED_PP(_Float16, 1), SPT_GROUPED_PP(_Float16, 2)},
      {SPT_GROUPED_PP(__bf16, 0), SPT_GROUPED_PP(__bf16, 1), SPT_GROUPED_PP(__bf16, 2)}};
#undef SPT_GROUPED_PP
  return fn[bf16][out];
}
GroupedEntry grouped_pp_entry(int mode, int bf16, int out) {
  const void* fn = mode == kGroupedForward ? pp_pick<kGroupedForward>(bf16, out)
                   : mode == kGroupedGradA ? pp_pick<kGroupedGradA>(bf16, out)
                                           : pp_pick<kGroupedGradB>(bf16, out);
  return GroupedEntry{fn, 256, 256, 512, 1};
}

}  // namespace spt
