// Shared definitions of the experts' operators: kernel arguments, and the search that maps a unit
// of work to the expert whose rows it covers.
//
// Rows sorted by expert are described by offsets[0 .. E] in device memory: expert e owns rows
// [offsets[e], offsets[e+1]). Rows before offsets[0] (some experts of an order) and from offsets[E] on
// belong to nobody. The counts are not known to the host, so a launch covers an upper bound of row blocks and
// every unit looks its expert up.
#pragma once

#include "spt_common.h"

namespace spt {

// Blocks of `bm` rows that E groups (and the rows behind the last, which the choice of a kernel counts on)
// can cut R rows into, at most: with g non-empty groups, (R - g) / bm + g. A launch covers one group more,
// the rows in front of the first.
SPT_HD int64_t max_row_blocks(int64_t rows, int64_t groups, int bm) {
  const int64_t g = groups + 1 < rows ? groups + 1 : rows;
  return rows <= 0 ? 0 : (rows - g) / bm + g;
}

struct GroupBlock {
  int e;       // the expert; E: rows of nobody; -1: no such unit
  int begin, end;  // the expert's rows
  int block;   // row block inside the expert
  int blocks;  // row blocks of the expert
  int local;   // unit number inside the expert
};

#if defined(__HIPCC__)
__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// Unit u's expert, where every block of `bm` rows holds `per` units: a wave reads 64 experts'
// offsets at once (one per lane), scans their unit counts, and finds the first lane whose running
// total passes u. All 64 lanes must be active. Offsets are clamped to [0, rows] and to ascending
// order inside an expert, so that no content of `offsets` leads outside the operands; a caller stops at the
// most units that ascending offsets can have, since experts whose rows overlap add up to more. With
// `rest`, the rows behind the last expert and those in front of the first are two more groups, e = E. The
// result is wave-uniform.
__device__ __forceinline__ GroupBlock find_group(const int* __restrict__ offsets, int E, int rows, int bm, int per,
                                                 bool rest, int u) {
  GroupBlock g;
  g.e = -1;
  g.begin = g.end = g.block = g.blocks = g.local = 0;
  int lane = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0));
  asm volatile("" : "+v"(lane));  // lane addresses are made here, not kept in registers across a caller's loop
  const int groups = rest ? E + 2 : E;
  int left = u;  // units still to skip
  for (int base = 0; base < groups; base += 64) {
    const int l = base + lane;
    int b = 0, en = 0;
    if (l < groups) {
      const int at = clampi(offsets[l <= E ? l : 0], 0, rows);
      b = l <= E ? at : 0;
      en = l < E ? clampi(offsets[l + 1], b, rows) : l == E ? rows : at;
    }
    const int nb = (int)((unsigned)(en - b + bm - 1) / (unsigned)bm);
    int s = nb * per;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(s, d);
      if (lane >= d) s += o;
    }
    const unsigned long long m = __ballot(s > left);
    if (m) {
      const int f = __builtin_ctzll(m);
      g.e = __builtin_amdgcn_readfirstlane(base + f < E ? base + f : E);
      g.begin = __builtin_amdgcn_readlane(b, f);
      g.end = __builtin_amdgcn_readlane(en, f);
      g.blocks = __builtin_amdgcn_readlane(nb, f);
      g.local = left - (__builtin_amdgcn_readlane(s, f) - g.blocks * per);
      g.block = g.local / per;
      return g;
    }
    left -= __builtin_amdgcn_readlane(s, 63);
  }
  return g;
}
#endif

// ------------------------------------------------------------------------------ sorted tokens
struct SortArgs {
  const void* ids;
  int id64;  // ids are 64-bit
  int rows;  // slots: tokens * top_k
  int experts;
  int per_block;  // slots of one workgroup (a multiple of 1024)
  int blocks;
  int* counts;  // [blocks][experts + 1], several workgroups only
  int* offsets;
  int* slots;
  int* rows_of;
};

struct RouteArgs {
  const char* src;  // rows read: x (gather), y (combine)
  const char* dout;  // combine's gradient
  char* dst;        // rows written: sorted rows, tokens, or the gradient of y
  const int* rows_of;   // [tokens][top_k] position of each slot among the sorted rows
  const int* kept;      // &offsets[E]
  const void* weights;  // [tokens][top_k], or null for ones
  void* dweights;
  int64_t ld_src, ld_dst, ld_dout;  // in elements
  int tokens, top_k, width;
  int lanes_log2;  // threads that share a token's row
  int zero_rest;
};

const void* sort_hist_fn();
const void* sort_place_fn();
const void* sort_one_fn();
// dtype 0 f16, 1 bf16, 2 f32; weight type: 0 .. 2, or 3 for none
const void* gather_fn(int dtype);
const void* combine_fn(int dtype, int wtype);
const void* combine_grad_fn(int dtype, int wtype);

// ------------------------------------------------------------------------------ grouped products
enum { kGroupedForward = 0, kGroupedGradA = 1, kGroupedGradB = 2 };

// D[i][j] = sum_c X[i][c] Y[j][c] per expert.
//   forward: X = A rows, Y = B[e] rows, c over K            (both contiguous in c)
//   grad A:  X = dC rows, Y[j][c] = B[e][c][j], c over N     (Y contiguous in j)
//   grad B:  X[i][c] = dC[c][i], Y[j][c] = A[c][j], c over the expert's rows (both contiguous in i, j)
struct GroupedArgs {
  const char* X;
  const char* Y;
  char* C;
  const int* offsets;
  int rows, experts;
  int m, n, kc;          // output rows (grad B only), output columns, contraction (not grad B)
  int64_t ldx, ldy, ldc;  // elements
  int64_t sy, sc;        // elements between experts in Y (forward, grad A) or C (grad B)
  int tiles_m, tiles_n;  // grad B: tiles of one expert; else tiles_n only
  int group_m;
  int grid;
  int units;             // output tiles (times parts of the sum) that ascending offsets make at most
  int rest;              // zero the output rows of nobody
  int nt;                // gradients, 256-row tiles: non-temporal stores
  int splits;            // 32-row tiles: parts of the sum, each into its fp32 plane at C (1: none)
  int64_t plane;         // elements between planes
};

struct PadArgs {
  const char* src;
  char* dst;
  int64_t rows, ld, rows_per, stride;  // row r is src + ((r / rows_per) * stride + (r % rows_per) * ld) elements
  int cols, cols_pad;
};

const void* pad_rows_fn();
struct GroupedEntry {
  const void* fn;
  int bm, bn, threads, per_cu;
};
// tile: rows of an output tile, 32 (not grad B), 128 or 256; deep: the 32-row tile's longer ring, Y streamed
GroupedEntry grouped_entry(int mode, int tile, bool deep, int bf16, int out);
GroupedEntry grouped_pp_entry(int mode, int bf16, int out);

// ------------------------------------------------------------------------------ 4-bit weights
struct W4PackArgs {
  const unsigned char* q;
  const unsigned short* scales;
  const unsigned char* zeros;
  char* packed;
  int64_t matrices;
  int n, k, group;
};

struct W4Args {
  const char* x;
  const char* w;       // packed blocks
  const char* scales;  // 16-bit, [matrix][n/16][k/128][16][128/group]
  const char* zeros;   // bytes, the same order
  char* out;           // output, or fp32 partial planes of a split sum
  const int* offsets;  // null: one matrix
  int64_t ldx, ldo;
  int64_t plane;       // elements between partial planes
  int rows, experts, n, k;
  int n16, kb;         // 16-column blocks, 128-deep blocks
  int splits;
  int rest;
  int out_dtype;
};

struct PlaneArgs {
  const float* parts;
  char* out;
  const int* offsets;  // rows that were computed: offsets[0] .. offsets[experts], or all when null
  int64_t ldo, plane;
  int rows, experts, n, splits, out_dtype;
};

struct W4Entry {
  const void* fn;
  int mt, nt, waves, wk;  // 16-row and 16-column blocks of a workgroup, its waves, and how many share out K
};
// variant 0, 1: 16 rows by 16 or 32 columns; sharing x, 2: 16 rows by 64; 3, 4: 32 rows by 64, 128; 5, 6: 64
// rows by 128, 256; 7: 16 rows by 128, fewer K parts than 2. gpk: groups per 128 k
W4Entry w4_entry(int variant, int bf16, int gpk, bool zero);
const void* w4_pack_fn();
const void* w4_pack_groups_fn();
const void* add_planes_fn();

}  // namespace spt
