// The experts' products over rows sorted by expert: C rows = A rows times their expert's B, and the
// gradients of both operands, in one kernel by the side on which each operand is contiguous.
//
//   D[i][j] = sum over c of X[i][c] * Y[j][c]
//   forward   X = A, Y = B[e]: both contiguous in c
//   grad A    X = dC (contiguous in c), Y[j][c] = B[e][c][j]: contiguous in j
//   grad B    X[i][c] = dC[c][i], Y[j][c] = A[c][j], c over the expert's rows: contiguous in i and j
//
// An operand that is contiguous in c is staged and read as in the dense kernels: rows of 64 c
// (128 bytes), chunk XOR (row mod 8), one ds_read_b128 per 16 x 32 fragment. One that is contiguous
// in i or j is staged as it lies, 64 rows of c by BM or BN columns, and turned on the way from LDS to
// registers (spt_transpose.h), so no transposed copy of B, A or dC is written to memory. Rows past an
// expert's last lie past its descriptor's end and read as zeros, so ragged experts need no padding in
// grad B's sum.
//
// Operands may start at any element and have rows of any length: a 16-byte load takes any byte offset. A
// chunk that reaches past the end of a row contiguous in c holds the next row's elements, which the last
// K-tile masks in both operands (0 * NaN is NaN); past the end of a row contiguous in i or j they meet only
// columns that are not stored. The descriptor's check drops a dword that is not wholly inside: with an odd
// row length it ends one element further, or, where that would lie past the operand itself, that one
// element is put into LDS by hand.
//
// A persistent grid walks the output tiles of all experts; each unit looks its expert up from the
// offsets (find_group), since the host does not know the counts. K-tiles of 64 stream through a ring
// of S LDS stages by direct global->LDS loads; one barrier per K-tile.
//
// Long sums of few tiles are cut into parts, each into its own fp32 plane, and a second kernel adds the planes in
// their order (32-row tiles only).
//
// What bounds it. Few rows per expert: reading B. 32 x 64 tiles keep 120 KiB of loads on the way per compute
// unit (two workgroups, five of six stages of 12 KiB; 108 KiB with three workgroups, three of four stages): 64
// rows, 8 experts of 4096 x 4096 in 44 us, 6.2 TB/s where every expert is met (a read-only stream reaches 5456
// GB/s; the rest are cache hits). More rows: 128 x 128 tiles, two workgroups a compute unit, whose
// barriers and waits overlap the other's products: 5003 rows, 64 experts of 1409 x 2044 (rows off 16 bytes, fp32
// out) 125 us, 3.3 TB/s and 230 TFLOP/s, where the loads' latency per K-tile (0.8 us for two tiles a compute unit)
// is what is left. Longer rings with one workgroup, 128 x 64 tiles and eight waves were no faster. From about 250
// rows per expert and enough tiles on the two-group kernel takes over (spt_grouped_pp.hip).
#include "spt_device.h"
#include "spt_experts.h"
#include "spt_transpose.h"

namespace spt {

// MODE: kGroupedForward .. ; a WM x WN grid of waves; S stages; PER_CU: workgroups per CU to fit; STREAM: Y
// loaded with the non-temporal hint.
template <int MODE, int BM, int BN, int WM, int WN, int S, int PER_CU, bool STREAM, typename TIn, int OUT>
__global__ void __launch_bounds__(64 * WM * WN, WM * WN * PER_CU / 4) grouped_kernel(GroupedArgs a) {
  constexpr bool TX = MODE == kGroupedGradB, TY = MODE != kGroupedForward;
  constexpr int W = WM * WN, BK = 64;
  constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  constexpr int XB = BM * BK * 2, YB = BN * BK * 2, STAGE = XB + YB;
  constexpr int LX = XB / 1024 / W, LY = YB / 1024 / W, LW = LX + LY;
  static_assert(XB % (1024 * W) == 0 && YB % (1024 * W) == 0, "every wave issues the same number of loads");
  static_assert(FM >= 1 && FN % 2 == 0 && S >= 2 && S * STAGE * PER_CU <= 160 * 1024, "tile");
  static_assert((S - 2) * LW < 64, "vmcnt is a 6-bit counter");
  __shared__ __attribute__((aligned(1024))) char smem[S * STAGE];
  const unsigned lds0 = lds_addr(smem);

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int p = lane & 15, h = lane >> 4;
  const int ldx = (int)a.ldx, ldy = (int)a.ldy, ldc = (int)a.ldc;
  constexpr int es = OUT == 2 ? 4 : 2;

  // load j of this wave: a lane's place in the operand tile. Contiguous in c: row and chunk of 8 c.
  // Contiguous in i or j: row c and chunk of 8 columns.
  const int n_kc = 8 * ((lane & 7) ^ swz(lane >> 3));
  // Y's row in LDS row r. 16-bit outputs: b_row_perm, so that a lane ends up with 8 consecutive output
  // columns per fragment pair, 16 bytes. fp32 outputs: as they lie; four consecutive columns are 16 bytes.
  auto y_row = [](int r) SPT_INLINE { return OUT == 2 ? r : b_row_perm(r); };
  auto x_off = [&](int j) SPT_INLINE {
    const int q = wave * LX + j;
    if constexpr (!TX) return (unsigned)((8 * q + (lane >> 3)) * ldx + n_kc) * 2u;
    else {
      const int c = q * (512 / BM) + lane / (BM / 8), ch = (lane % (BM / 8)) ^ (2 * tr_swz<BM>(c));
      return (unsigned)(c * ldx + 8 * ch) * 2u;
    }
  };
  auto y_off = [&](int j) SPT_INLINE {
    const int q = wave * LY + j;
    if constexpr (!TY) return (unsigned)(y_row(8 * q + (lane >> 3)) * ldy + n_kc) * 2u;
    else {
      const int c = q * (512 / BN) + lane / (BN / 8), ch = (lane % (BN / 8)) ^ (2 * tr_swz<BN>(c));
      return (unsigned)(c * ldy + 8 * ch) * 2u;
    }
  };

  // fragment f of k-step s
  auto read_x = [&](const char* t, int s, int f) SPT_INLINE -> u32x4 {
    if constexpr (!TX) return *(const u32x4*)(t + lds_chunk_offset(BM, wm * TM + 16 * f + p, 4 * s + h));
    else return tr_frag<2 * BM>(t + tr_offset<BM>(32 * s + 8 * h + (p >> 2), (wm * TM + 16 * f) / 16) + 8 * (p & 3));
  };
  auto read_y = [&](const char* t, int s, int f) SPT_INLINE -> u32x4 {
    if constexpr (!TY) return *(const u32x4*)(t + lds_chunk_offset(BN, wn * TN + 16 * f + p, 4 * s + h));
    else return tr_frag<2 * BN>(t + tr_offset<BN>(32 * s + 8 * h + (p >> 2), (wn * TN + 16 * f) / 16) + 8 * (p & 3));
  };

  constexpr bool kSplit = BM == 32;
  for (int tp = xcd_remap(blockIdx.x, a.grid); tp < a.units; tp += a.grid) {
    // this unit: output tile (row0, col0), its row and column counts, the sum's length and its part of it
    int e, row0, rows_left, tm, tn, kc, c0 = 0, part = 0;
    int t = tp;
    if constexpr (kSplit) {
      t = tp / a.splits;
      part = tp - t * a.splits;
    }
    if constexpr (MODE == kGroupedGradB) {
      const int per = a.tiles_m * a.tiles_n;
      e = t / per;
      grouped_raster(t - e * per, a.tiles_m, a.tiles_n, a.group_m, tm, tn);
      row0 = tm * BM;
      rows_left = a.m - row0;
      c0 = clampi(a.offsets[e], 0, a.rows);
      kc = clampi(a.offsets[e + 1], c0, a.rows) - c0;
      c0 = __builtin_amdgcn_readfirstlane(c0);
      kc = __builtin_amdgcn_readfirstlane(kc);
    } else {
      const GroupBlock g = find_group(a.offsets, a.experts, a.rows, BM, a.tiles_n, a.rest != 0, t);
      if (g.e < 0) break;
      e = g.e;
      grouped_raster(g.local, g.blocks, a.tiles_n, a.group_m, tm, tn);
      row0 = g.begin + tm * BM;
      rows_left = g.end - row0;
      kc = e == a.experts ? 0 : a.kc;  // rows of nobody: zeros
    }
    const int col0 = tn * BN, cols_left = a.n - col0;
    const char* xb = a.X + (MODE == kGroupedGradB ? ((int64_t)c0 * a.ldx + row0) * 2 : (int64_t)row0 * a.ldx * 2);
    const char* yb = a.Y + (MODE == kGroupedGradB ? ((int64_t)c0 * a.ldy + col0) * 2
                            : MODE == kGroupedGradA ? ((int64_t)e * a.sy + col0) * 2
                                                    : ((int64_t)e * a.sy + (int64_t)col0 * a.ldy) * 2);
    // Odd row lengths: the descriptor ends one element further (more = 1), but in the tile that holds the
    // operand's very last element (patch). In whole-number arithmetic, which stays in scalar registers.
    auto at_most_1 = [](int v) SPT_INLINE { return v < 1 ? (v < 0 ? 0 : v) : 1; };
    const int x_behind = MODE == kGroupedGradB ? a.rows - c0 - kc : a.rows - row0 - rows_left;
    const int y_behind = MODE == kGroupedGradB ? a.rows - c0 - kc : a.experts - 1 - e;
    const int x_more = (TX ? rows_left : kc) & (at_most_1(x_behind) | at_most_1(rows_left - BM));
    const int y_more = (TY ? cols_left : kc) & (at_most_1(y_behind) | at_most_1(cols_left - BN));
    const bool x_patch = ((TX ? rows_left : kc) & 1) != x_more, y_patch = ((TY ? cols_left : kc) & 1) != y_more;
    // K-tiles first .. first + kt - 1; `end`: where the part's K-tiles end (or the sum)
    const int all = (kc + BK - 1) / BK, per = kSplit ? (all + a.splits - 1) / a.splits : all, first = part * per;
    const int kt = all - first < per ? (all - first < 0 ? 0 : all - first) : per;
    const int end = (first + kt) * BK < kc ? (first + kt) * BK : kc;
    const bool last_part = first + kt == all;
    auto issue = [&](int i) SPT_INLINE {
      const int k0 = (first + i) * BK;
      const unsigned dst = lds0 + (unsigned)(i % S) * STAGE;
      // K-tiles past the end read nothing and fill zeros, so every K-tile issues LW loads
      auto rsrc = [&](bool tr, const char* base, int64_t ld, int rows, int width, int odd) SPT_INLINE {
        const int some = end > k0;
        const int64_t left = some ? (tr ? kc - k0 : rows) : 1;  // memory rows that may be read
        const int64_t bytes = ((left - 1) * ld + width + odd) * 2 * some;
        return make_rsrc(base + (tr ? (int64_t)k0 * ld * 2 : 0), (uint64_t)bytes);
      };
      const __amdgpu_buffer_rsrc_t rx = rsrc(TX, xb, a.ldx, rows_left, TX ? rows_left : kc, x_more);
      const __amdgpu_buffer_rsrc_t ry = rsrc(TY, yb, a.ldy, cols_left, TY ? cols_left : kc, y_more);
#pragma unroll
      for (int j = 0; j < LX; ++j) {
        const unsigned v = x_off(j);
        dma16_unseen(rx, dst + (wave * LX + j) * 1024, TX || n_kc < kc - k0 ? v : kOOB, TX ? 0u : 2u * k0);
      }
#pragma unroll
      for (int j = 0; j < LY; ++j) {
        const unsigned v = y_off(j);
        const unsigned at = dst + XB + (wave * LY + j) * 1024, voff = TY || n_kc < kc - k0 ? v : kOOB;
        if constexpr (STREAM) dma16_unseen_stream(ry, at, voff, TY ? 0u : 2u * k0);
        else dma16_unseen(ry, at, voff, TY ? 0u : 2u * k0);
      }
    };

    f32x4 acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // K-tile k's products, from its stage. kCut: the K-tile reaches past kc, whose elements from there on are
    // masked in operands contiguous in c.
    auto products = [&](int k, auto cut_c) SPT_INLINE {
      constexpr bool kCut = decltype(cut_c)::value;
      const char* xt = smem + (k % S) * STAGE;
      const char* yt = xt + XB;
#pragma unroll
      for (int s = 0; s < BK / 32; ++s) {
        u32x4 xf[FM], yf[FN];
#pragma unroll
        for (int f = 0; f < FN; ++f) yf[f] = read_y(yt, s, f);
#pragma unroll
        for (int f = 0; f < FM; ++f) xf[f] = read_x(xt, s, f);
        if constexpr (kCut) {
          const int left = kc - (first + k) * BK - 32 * s - 8 * h;  // elements of the lane's eight that exist
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const unsigned keep = left >= 2 * w + 2 ? ~0u : (left == 2 * w + 1 ? 0xFFFFu : 0u);
            if constexpr (!TY) {
#pragma unroll
              for (int f = 0; f < FN; ++f) yf[f][w] &= keep;
            }
            if constexpr (!TX) {
#pragma unroll
              for (int f = 0; f < FM; ++f) xf[f][w] &= keep;
            }
          }
        }
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
          for (int j = 0; j < FM; ++j) acc[i][j] = mfma16<TIn>(yf[i], xf[j], acc[i][j]);
      }
    };
    // an operand's very last element, which no load reaches (see the top), into its place in stage `st`
    auto patch = [&](int st) SPT_INLINE {
      const int c = kc - 1 - (all - 1) * BK;
      char* xt = smem + st * STAGE;
      if (x_patch && threadIdx.x == 0) {
        const int r = rows_left - 1;
        const int64_t at = TX ? (int64_t)(kc - 1) * a.ldx + r : (int64_t)r * a.ldx + kc - 1;
        const int o = TX ? tr_offset<TX ? BM : 128>(c, r >> 4) + 2 * (r & 15) : lds_chunk_offset(BM, r, c >> 3) + 2 * (c & 7);
        *(unsigned short*)(xt + o) = *(const unsigned short*)(xb + 2 * at);
      }
      if (y_patch && threadIdx.x == 64) {
        const int r = cols_left - 1;
        const int64_t at = TY ? (int64_t)(kc - 1) * a.ldy + r : (int64_t)r * a.ldy + kc - 1;
        // b_row_perm's LDS row of row 8 g + 4 h + i is 16 h + 4 g + i
        const int lr = OUT == 2 ? r : (r & ~31) + 16 * ((r >> 2) & 1) + 4 * ((r >> 3) & 3) + (r & 3);
        const int o = TY ? tr_offset<BN>(c, r >> 4) + 2 * (r & 15) : lds_chunk_offset(BN, lr, c >> 3) + 2 * (c & 7);
        *(unsigned short*)(xt + XB + o) = *(const unsigned short*)(yb + 2 * at);
      }
      wait_lgkmcnt0();
      barrier_sync();
    };
    wait_vmcnt<0>();  // the previous unit's loads past its end, and its stores
    barrier_sync();   // ... and everybody's reads of the ring
    if (kt > 0) {
#pragma unroll
      for (int s = 0; s < S - 1; ++s) issue(s);
      for (int k = 0; k < kt - 1; ++k) {
        wait_vmcnt<(S - 2) * LW>();  // K-tile k has landed: only later ones in flight
        barrier_sync();              // for every wave; and K-tile k - 1 has been read by all
        issue(k + S - 1);
        products(k, std::false_type{});
      }
      wait_vmcnt<(S - 2) * LW>();
      barrier_sync();
      if (last_part && (x_patch || y_patch)) patch((kt - 1) % S);
      if ((!TX || !TY) && last_part && (kc & 7)) products(kt - 1, std::true_type{});
      else products(kt - 1, std::false_type{});
    }

    const __amdgpu_buffer_rsrc_t rc = make_rsrc(
        a.C + ((MODE == kGroupedGradB ? (int64_t)e * a.sc : 0) + (kSplit ? part * a.plane : 0) + (int64_t)row0 * a.ldc) * es,
        ((uint64_t)(rows_left - 1) * a.ldc + a.n) * es);
    const bool full = rows_left >= BM && cols_left >= BN;
    if constexpr (OUT == 2) {
#pragma unroll
      for (int j = 0; j < FM; ++j) {
#pragma unroll
        for (int i = 0; i < FN; ++i) {
          const int m = wm * TM + 16 * j + p, n = col0 + wn * TN + 16 * i + 4 * h;
          if (full) store4_f32<false>(acc[i][j], rc, m, rows_left, n, a.n, ldc);
          else store4_f32<true>(acc[i][j], rc, m, rows_left, n, a.n, ldc);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      continue;
    }
#pragma unroll
    for (int j = 0; j < FM; ++j) {
#pragma unroll
      for (int pu = 0; pu < FN / 2; ++pu) {
        float v[8];
        if constexpr (TY) {
          pair_columns(acc[2 * pu][j], acc[2 * pu + 1][j], v);
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            v[q] = acc[2 * pu][j][q];
            v[4 + q] = acc[2 * pu + 1][j][q];
          }
        }
        const int m = wm * TM + 16 * j + p, n = col0 + wn * TN + 32 * pu + (TY ? pair_column(lane) : 8 * h);
        if (full) store8<OUT, false>(v, rc, m, rows_left, n, a.n, ldc);
        else store8<OUT, true>(v, rc, m, rows_left, n, a.n, ldc);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  wait_vmcnt<0>();  // no load may still be on its way to LDS when the workgroup ends
}

// ------------------------------------------------------------------------------ padding
// Operands whose rows are not 16-byte aligned multiples of 8 elements are copied to rows that are,
// the padding columns zero: the direct loads move whole 16-byte chunks.
__global__ void __launch_bounds__(256) pad_rows_kernel(PadArgs a) {
  typedef unsigned u32x4u __attribute__((ext_vector_type(4), aligned(2)));
  const int cpr = a.cols_pad / 8;
  const int64_t total = a.rows * cpr;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / cpr;
    const int col = (int)(i - r * cpr) * 8;
    const char* s = a.src + ((r / a.rows_per) * a.stride + (r % a.rows_per) * a.ld + col) * 2;
    u32x4 v = {0, 0, 0, 0};
    if (col + 8 <= a.cols) {
      v = *(const u32x4u*)s;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (col + e < a.cols) v[e >> 1] |= (unsigned)((const unsigned short*)s)[e] << (16 * (e & 1));
    }
    *(u32x4*)(a.dst + i * 16) = v;
  }
}
const void* pad_rows_fn() { return (const void*)&pad_rows_kernel; }

// ------------------------------------------------------------------------------ instantiations
template <int MODE, int BM, int BN, int WM, int WN, int S, int PER_CU, bool STREAM = false>
static GroupedEntry grouped_pick(int bf16, int out) {
  GroupedEntry e{nullptr, BM, BN, 64 * WM * WN, PER_CU};
#define SPT_GROUPED(TI, O) (const void*)&grouped_kernel<MODE, BM, BN, WM, WN, S, PER_CU, STREAM, TI, O>
  static const void* const fn[2][3] = {{SPT_GROUPED(_Float16, 0), SPT_GROUPED(_Float16, 1), SPT_GROUPED(_Float16, 2)},
                                       {SPT_GROUPED(__bf16, 0), SPT_GROUPED(__bf16, 1), SPT_GROUPED(__bf16, 2)}};
#undef SPT_GROUPED
  e.fn = fn[bf16][out];
  return e;
}
GroupedEntry grouped_entry(int mode, int tile, bool deep, int bf16, int out) {
  if (tile == 256) return grouped_pp_entry(mode, bf16, out);
  if (mode == kGroupedForward)
    return tile == 128 ? grouped_pick<kGroupedForward, 128, 128, 2, 2, 2, 2>(bf16, out)
           : deep      ? grouped_pick<kGroupedForward, 32, 64, 2, 2, 6, 2, true>(bf16, out)
                       : grouped_pick<kGroupedForward, 32, 64, 2, 2, 4, 3>(bf16, out);
  if (mode == kGroupedGradA)
    return tile == 128 ? grouped_pick<kGroupedGradA, 128, 128, 2, 2, 2, 2>(bf16, out)
           : deep      ? grouped_pick<kGroupedGradA, 32, 64, 2, 2, 6, 2, true>(bf16, out)
                       : grouped_pick<kGroupedGradA, 32, 128, 2, 2, 4, 2>(bf16, out);  // B's rows are c: longer pieces
  return grouped_pick<kGroupedGradB, 128, 128, 2, 2, 2, 2>(bf16, out);
}

}  // namespace spt
