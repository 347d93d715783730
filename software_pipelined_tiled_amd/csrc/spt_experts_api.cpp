// Host side of include/experts.h: argument checks, the choice of a kernel, launches. Nothing here
// allocates or synchronises, and no state outlives a call but the devices' properties.
#include <cstring>
#include <mutex>

#include "experts.h"
#include "spt_experts.h"

namespace {

constexpr int64_t kMax32 = 0x7FFFFFFF;
constexpr int kMaxExperts = 1024;  // of the sort, whose workgroups count in LDS
constexpr int64_t kMaxGroups = (int64_t)1 << 24;  // of the products: the search adds 64 to their number in 32 bits
// Output tiles of a grouped product: 64 experts' counts add up in 32 bits whatever the offsets hold. Of the
// smallest tiles these are 2^35 elements.
constexpr int64_t kMaxUnits = (int64_t)1 << 24;
constexpr int kMaxDevices = 64;
// Bytes of one operand: byte counts and offsets stay inside 64 bits, and no memory is as large.
constexpr int64_t kMaxBytes = (int64_t)1 << 56;
constexpr int64_t kMaxGridY = 65535;
constexpr int kCus = 256;  // the MI355X's, for choices that must not depend on the device in use

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }
bool is16(gemm_dtype_t d) { return d == GEMM_F16 || d == GEMM_BF16; }
bool is_dtype(gemm_dtype_t d) { return is16(d) || d == GEMM_F32; }

// Compute units of the current device; GEMM_ERR_HIP unless it is a gfx950.
gemm_status_t device_cus(int* cu) {
  static std::mutex mu;
  static int known[kMaxDevices];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) {
    (void)hipGetLastError();
    return GEMM_ERR_HIP;
  }
  if (dev < 0 || dev >= kMaxDevices) return GEMM_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(mu);
  if (known[dev] == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
      (void)hipGetLastError();
      return GEMM_ERR_HIP;
    }
    if (std::strncmp(prop.gcnArchName, "gfx950", 6) != 0) return GEMM_ERR_HIP;
    known[dev] = prop.multiProcessorCount;
  }
  *cu = known[dev];
  return GEMM_OK;
}

gemm_status_t launch(const void* fn, dim3 grid, int threads, int lds, void* arg, void* stream) {
  void* kargs[] = {arg};
  if (hipLaunchKernel(fn, grid, dim3(threads), kargs, lds, (hipStream_t)stream) != hipSuccess) {
    (void)hipGetLastError();
    return GEMM_ERR_HIP;
  }
  return GEMM_OK;
}

int stream_grid(int64_t threads) {
  const int64_t b = ceil_div(threads, 256);
  return (int)(b < 1 ? 1 : (b > 8192 ? 8192 : b));
}

// out = the planes of a cut sum, added in their order; with offsets, the experts' rows only
gemm_status_t add_planes(const float* parts, void* out, const int32_t* offsets, int64_t experts, int64_t ldo, int64_t rows,
                         int64_t n, int64_t splits, int out_dtype, void* stream) {
  spt::PlaneArgs r;
  r.parts = parts;
  r.out = (char*)out;
  r.offsets = offsets;
  r.ldo = ldo;
  r.plane = rows * n;
  r.rows = (int)rows;
  r.experts = (int)experts;
  r.n = (int)n;
  r.splits = (int)splits;
  r.out_dtype = out_dtype;
  return launch(spt::add_planes_fn(), dim3(stream_grid(r.plane)), 256, 0, &r, stream);
}

// ---------------------------------------------------------------------------------- sort
// One workgroup sorts up to kSortOne slots by itself (4096 slots of 64 experts: 6.7 us in one launch, 6.9 in
// two; 8192: 10.5 against 6.9); beyond, each workgroup takes kSortBlock of them
// (more when there would be over 256 workgroups, since each adds up every other's counts).
constexpr int64_t kSortOne = 4096, kSortBlock = 1024;
struct SortShape {
  int64_t per_block, blocks;
};
SortShape sort_shape(int64_t slots) {
  if (slots <= kSortOne) return {slots, 1};
  int64_t per = round_up(ceil_div(slots, 256), 1024);
  if (per < kSortBlock) per = kSortBlock;
  return {per, ceil_div(slots, per)};
}

gemm_status_t check_route(gemm_dtype_t dtype, int64_t tokens, int64_t top_k, int64_t width) {
  if (!is_dtype(dtype) || tokens < 0 || top_k < 0 || width < 0) return GEMM_ERR_INVALID;
  if (tokens > kMax32 || top_k > kMax32 || width > kMax32 || tokens * top_k > kMax32) return GEMM_ERR_UNSUPPORTED;
  return GEMM_OK;
}

// Threads per token: the power of two that covers the row's 16-byte chunks, at most a workgroup.
gemm_status_t route_grid(int64_t tokens, int64_t width, int* lanes_log2, dim3* grid) {
  const int64_t chunks = ceil_div(width, 8);
  int l = 0;
  while (l < 8 && ((int64_t)1 << l) < chunks) ++l;
  const int64_t gx = ceil_div(tokens, 256 >> l), gy = ceil_div(chunks, (int64_t)1 << l);
  if (gx * 256 > kMax32 || gy > kMaxGridY) return GEMM_ERR_UNSUPPORTED;
  *lanes_log2 = l;
  *grid = dim3((unsigned)gx, (unsigned)gy);
  return GEMM_OK;
}

// ---------------------------------------------------------------------------------- grouped
struct Operand {
  int64_t rows, cols, ld, rows_per, stride;  // rows of a matrix per expert; stride between experts
  bool pad;                                  // copied to the workspace
  int64_t pad_ld, at, bytes;
};
struct GroupedShape {
  int tile;
  Operand x, y;
  int64_t splits, planes, ws;  // parts of a sum; where their planes begin in the workspace
};

// 32-row tiles: with at most two of them for every compute unit and rows of whole 16-byte chunks, two
// workgroups of six stages, five in flight, and the hint that keeps Y, which is read once then, out of the caches
// (64 rows, 8 experts, 4096^2: 44 us against 57 with three workgroups of four stages, three in flight). With more
// tiles a third workgroup saves a round (200 rows: 59 against 77), and off 16 bytes neighbouring loads share lines,
// and the hint costs (2044 columns: 56 us against 49).
int64_t grouped_small_tiles(const gemm_grouped_t* p) {
  const int64_t out_n = p->mode == GEMM_GROUPED_FORWARD ? p->n : p->k;
  const int64_t used = p->experts < p->rows ? p->experts : p->rows;
  const int64_t blocks = used + (p->rows > 16 * used ? (p->rows - 16 * used) / 32 : 0);  // about
  return blocks * ceil_div(out_n, 64);
}
bool grouped_few(const gemm_grouped_t* p) { return grouped_small_tiles(p) <= 2 * kCus; }
bool grouped_deep(const gemm_grouped_t* p, const void* Y) {
  return grouped_few(p) && (uintptr_t)Y % 16 == 0 && p->k % 8 == 0 && p->ldy % 8 == 0;
}

// Rows of an output tile: the least time by this model, in us. A start, and the longer of rounds of tiles over the
// compute units (K-tiles times what one takes, and the tile's own start and end) and the operands' bytes.
// 256-row tiles copy an operand that is off 16 bytes first. The constants are a fit to 1608 measured shapes
// (1 .. 128 experts, 32 .. 16384 rows, N and K 512 .. 8192); on them the choice takes 2 % longer than the best tile of
// each shape, 47 % at worst, where 32-row tiles for up to 32 rows per expert and rounds alone took 7 %, 185 % at
// worst (grad B of 64 experts of 1001 x 1500, 32 rows: 113 us against 39). On 414 other shapes, drawn at random
// with uneven experts, it takes 2.9 %, 73 % at worst (3230 rows, one expert of 5249 x 7795: 585 us against 338).
//   Two things the model leaves out. Grad A's 32-row tiles beyond two for every compute unit read B in pieces of 256
// bytes from many places, and 128-row tiles are faster even for few rows (128 rows, 16 experts, 4096^2: 86 us against
// 94). And grad B's 128-row tiles reload what the L2 no longer holds from about 64 rows per expert on (16384
// rows, 128 experts, 2048 x 512: 150 us, the model says 93); with long sums that hides behind the products.
int grouped_tile(const gemm_grouped_t* p, const Operand* const (&ops)[2], const bool (&off)[2]) {
  const bool gb = p->mode == GEMM_GROUPED_GRAD_B, fwd = p->mode == GEMM_GROUPED_FORWARD;
  const int64_t used = p->experts < p->rows ? p->experts : p->rows;
  if (used == 0) return 128;
  const int64_t out_n = fwd ? p->n : p->k;
  const double rows = (double)p->rows, n = (double)p->n, k = (double)p->k;
  const double mb = ((double)(gb ? p->experts : used) * n * k + rows * (n + k)) * 2e-6;
  const double each = rows / (double)p->experts;
  // an expert's last K-tile (grad B) or row block is half full on average
  const double kt = gb ? each / 64 + 0.5 : (double)ceil_div(fwd ? p->k : p->n, 64);
  double copy = 0;
  for (int i = 0; i < 2; ++i)
    if (off[i]) copy += 3 + (double)ops[i]->rows * (double)ops[i]->cols * 4 / 4.5e6;  // read and written at 4.5 TB/s
  struct Tile {
    int bm, bn, slots;
    struct { double start, k_tile, tile, mb; } by_mode[3];
  };
  static const Tile tiles[3] = {
      {32, 64, 3 * kCus, {{1.0, .41, 4.7, .17}, {1.4, .49, 4.1, .19}, {}}},
      {128, 128, 2 * kCus, {{0, .77, 6.0, .21}, {0, .78, 6.2, .19}, {5.8, .87, 3.2, .19}}},
      {256, 256, kCus, {{0, 1.07, 7.8, .23}, {0, 1.2, 9.4, .22}, {4.0, 1.5, 6.3, .28}}}};
  int best = 0;
  double least = 0;
  for (const Tile& t : tiles) {
    if (t.bm == 32 && (gb || (!fwd && !grouped_few(p)))) continue;
    const auto& c = t.by_mode[p->mode];
    int64_t rb = gb ? p->experts * ceil_div(p->n, t.bm) : (2 * p->rows + used * t.bm) / (2 * t.bm);
    if (rb < used) rb = used;
    const double work = (double)ceil_div(rb * ceil_div(out_n, t.bn), t.slots) * (c.k_tile * kt + c.tile);
    double us = c.start + (work > c.mb * mb ? work : c.mb * mb);
    if (t.bm == 256) us += copy;
    if (t.bm == 128 && gb && each >= 64 && each < 512) us *= 1.2;
    if (best == 0 || us < least) best = t.bm, least = us;
  }
  return best;
}

gemm_status_t grouped_shape(const gemm_grouped_t* p, const void* X, const void* Y, GroupedShape* s) {
  if (!p || p->mode < GEMM_GROUPED_FORWARD || p->mode > GEMM_GROUPED_GRAD_B) return GEMM_ERR_INVALID;
  if (p->rows < 0 || p->experts < 0 || p->n < 0 || p->k < 0) return GEMM_ERR_INVALID;
  if (!is_dtype(p->in_dtype) || !is_dtype(p->out_dtype)) return GEMM_ERR_INVALID;
  if (p->tile != 0 && p->tile != 32 && p->tile != 128 && p->tile != 256) return GEMM_ERR_INVALID;
  if (!is16(p->in_dtype) || (p->tile == 32 && p->mode == GEMM_GROUPED_GRAD_B)) return GEMM_ERR_UNSUPPORTED;
  const int64_t lim = (int64_t)1 << 20;
  if (p->rows > kMax32 || p->experts > kMaxGroups || p->n > kMax32 || p->k > kMax32) return GEMM_ERR_UNSUPPORTED;
  const bool gb = p->mode == GEMM_GROUPED_GRAD_B;
  const int64_t xc = p->mode == GEMM_GROUPED_FORWARD ? p->k : p->n;
  const int64_t oc = p->mode == GEMM_GROUPED_FORWARD ? p->n : p->k;
  if (p->ldx < xc || p->ldy < p->k || p->ldo < oc) return GEMM_ERR_INVALID;
  if (p->ldx >= lim || p->ldy >= lim || p->ldo >= lim) return GEMM_ERR_UNSUPPORTED;
  const int64_t mat_ld = gb ? p->ldo : p->ldy;  // of the [experts, n, k] tensor
  const int64_t span = p->n > 0 ? (p->n - 1) * mat_ld + p->k : 0;
  if (p->experts > 1 && p->stride < span) return GEMM_ERR_INVALID;
  if (p->experts > 0 && (p->stride > span ? p->stride : span) > kMaxBytes / 4 / p->experts) return GEMM_ERR_UNSUPPORTED;
  s->x = Operand{p->rows, xc, p->ldx, p->rows > 0 ? p->rows : 1, 0, false, 0, 0, 0};
  if (gb) s->y = Operand{p->rows, p->k, p->ldy, p->rows > 0 ? p->rows : 1, 0, false, 0, 0, 0};
  else s->y = Operand{p->experts * p->n, p->k, p->ldy, p->n > 0 ? p->n : 1, p->stride, false, 0, 0, 0};
  s->ws = 0;
  Operand* const ops[2] = {&s->x, &s->y};
  const void* ptr[2] = {X, Y};
  bool off[2];  // not in rows of whole 16-byte chunks
  for (int i = 0; i < 2; ++i)
    off[i] = (uintptr_t)ptr[i] % 16 != 0 || ops[i]->cols % 8 != 0 || ops[i]->ld % 8 != 0 || ops[i]->stride % 8 != 0;
  s->tile = p->tile ? p->tile : grouped_tile(p, {ops[0], ops[1]}, off);
  for (int i = 0; i < 2; ++i) {
    Operand& o = *ops[i];
    o.pad = s->tile == 256 && off[i];
    if (!o.pad) continue;
    o.pad_ld = round_up(o.cols, 8);
    o.at = s->ws;
    o.bytes = round_up(o.rows * o.pad_ld * 2, 256);
    s->ws += o.bytes;
  }
  // 32-row tiles that fill less than half of two to a compute unit: parts of the sum of eight K-tiles or more, as
  // many as run at once, where that spares a workgroup 18 K-tiles (5 us; the second pass costs 4): 2 rows, 8 experts
  // of 4096^2 21 -> 18.5 us, of 4096 x 14336 67 -> 43, 1 row of 4096^2 20 -> 14; but 2 rows of 4096 x 1536, three
  // parts, 11.1 -> 11.6, and 8 rows, 64 experts of 1408 x 2048, two parts, 14 -> 16.
  s->splits = 1;
  s->planes = s->ws;
  if (s->tile == 32 && p->rows > 0) {
    const int64_t tiles = grouped_small_tiles(p), kt = ceil_div(p->mode == GEMM_GROUPED_FORWARD ? p->k : p->n, 64);
    if (tiles > 0) {
      const int64_t fit = 2 * kCus / tiles, most = kt / 8;
      s->splits = fit < most ? fit : most;
      if (s->splits < 2 || kt - kt / s->splits < 18) s->splits = 1;
      else s->ws += s->splits * p->rows * oc * 4;
    }
  }
  return GEMM_OK;
}

gemm_status_t pad_operand(Operand& o, const void** ptr, char* ws, void* stream) {
  if (!o.pad || o.rows == 0 || o.cols == 0) return GEMM_OK;
  spt::PadArgs a;
  a.src = (const char*)*ptr;
  a.dst = ws + o.at;
  a.rows = o.rows; a.ld = o.ld; a.rows_per = o.rows_per; a.stride = o.stride;
  a.cols = (int)o.cols; a.cols_pad = (int)o.pad_ld;
  const gemm_status_t st = launch(spt::pad_rows_fn(), dim3(stream_grid(o.rows * (o.pad_ld / 8))), 256, 0, &a, stream);
  *ptr = a.dst;
  o.ld = o.pad_ld;
  if (o.stride) o.stride = o.rows_per * o.pad_ld;
  return st;
}

// ---------------------------------------------------------------------------------- 4-bit weights
int64_t w4_blocks(int64_t matrices, int64_t n, int64_t k) { return matrices * ceil_div(n, 16) * ceil_div(k, 128); }

// n and k up to 2^24 leave a matrix up to 2^37 blocks, of at most 1024 + 16 * 4 * 3 bytes
bool w4_too_large(int64_t matrices, int64_t n, int64_t k) {
  const int64_t each = w4_blocks(1, n, k);
  return each > 0 && matrices > kMaxBytes / 2048 / each;
}

struct W4Shape {
  spt::W4Entry entry;
  int64_t nblocks, row_blocks, grid_y, splits, ws;  // row_blocks: what the choice counts on
};

gemm_status_t w4_shape(const gemm_w4_t* p, bool grouped, W4Shape* s) {
  if (!p || p->rows < 0 || p->matrices < 0 || p->n < 0 || p->k < 0) return GEMM_ERR_INVALID;
  if (!is_dtype(p->dtype) || !is_dtype(p->out_dtype)) return GEMM_ERR_INVALID;
  if (!is16(p->dtype) || (p->group != 32 && p->group != 64 && p->group != 128)) return GEMM_ERR_UNSUPPORTED;
  if (p->ldx < p->k || p->ldo < p->n || (!grouped && p->matrices != 1)) return GEMM_ERR_INVALID;
  const int64_t lim = (int64_t)1 << 24;
  if (p->n > lim || p->k > lim || p->ldx >= lim / 2 || p->rows > kMax32 || p->matrices > kMaxGroups ||
      w4_too_large(p->matrices, p->n, p->k))
    return GEMM_ERR_UNSUPPORTED;
  const int64_t n16 = ceil_div(p->n, 16), kb = ceil_div(p->k, 128);
  const int64_t each = p->matrices > 0 ? ceil_div(p->rows, p->matrices) : 0;  // rows that share a matrix, on average
  const int64_t used = p->rows < p->matrices ? p->rows : p->matrices;
  auto take = [&](int variant) {
    s->entry = spt::w4_entry(variant, p->dtype == GEMM_BF16, 128 / p->group, p->has_zeros != 0);
    s->nblocks = ceil_div(n16, s->entry.nt);
    const int bm = 16 * s->entry.mt;
    s->row_blocks = grouped ? spt::max_row_blocks(p->rows, p->matrices, bm) : ceil_div(p->rows, bm);
    s->grid_y = grouped ? spt::max_row_blocks(p->rows, p->matrices + 1, bm) : s->row_blocks;
  };
  // Cut K when the workgroups alone leave compute units idle, into as many parts as still run at once: one
  // workgroup more than compute units is a second round.
  auto splits = [&]() {
    const int64_t wgs = s->nblocks * s->row_blocks, most = kb / s->entry.waves;
    if (wgs <= 0 || wgs >= kCus) return (int64_t)1;
    const int64_t n = kCus / wgs < most ? kCus / wgs : most;
    return n < 1 ? (int64_t)1 : n;
  };
  // Many blocks of up to 16 rows with short sums: few K parts (64 experts of 1408 x 2048, 64 rows: 21 us
  // against 25 to 59; 16 of 2048 x 2048, 8 rows: 9.7 against 7.4). Up to four rows a matrix: the waves take K
  // slices straight from memory, 16 columns to a workgroup where that fills the compute units at most once
  // (4096 x 4096, 1 row: 5.0 us, 32 columns 6.6; 8192 x 8192: 13.0 against 10.3). Else the least time by this
  // model, in us: a start, rounds of workgroups over the compute units times blocks of K per wave, and the second
  // pass over a split sum. Its constants are a fit to 1320 measured shapes (N 512 .. 28672, K 1024 .. 14336, 1 ..
  // 2000 rows, up to 64 experts). On them the choice takes 2 % longer than the best kernel of each shape, 39 % at
  // worst; a rule on the number of 16 x 16 output blocks alone took 9 %, 95 % at worst. On 132 other shapes, drawn at
  // random with uneven experts, it takes 9 %, 62 % at worst (290 rows over 26 experts of 539 x 13773: 92 us against
  // 57), most of it where the model's candidates leave out the kernels of the two rules before it.
  // Blocks of rows are the grid's second dimension: where a kernel's are too many, only those with more rows a block
  // are candidates.
  int chosen = -1;
  if (each <= 16 && kb <= 16 && p->matrices > 1 && n16 * used >= 1536) chosen = 7;
  else if (each <= 4) chosen = n16 * used <= kCus ? 0 : 1;
  if (chosen >= 0) take(chosen);
  if (chosen < 0 || s->grid_y > kMaxGridY) {
    struct { double start, block, extra; } const t[] = {
        {3.9, 1.03, 0.7}, {3.5, .82, 1.6}, {3.4, 1.19, 1.8}, {4.8, .96, 1.4}, {5.3, .73, 1.9}, {3.4, 1.27, 3.1}};
    int best = 0;
    double least = 0;
    for (int v = 1; v <= 6; ++v) {
      take(v);
      if (s->grid_y > kMaxGridY) continue;
      const int64_t sp = splits(), wgs = s->nblocks * used * ceil_div(each, 16 * s->entry.mt) * sp;
      const double blocks = (double)ceil_div(ceil_div(kb, sp), s->entry.wk);
      const double us = t[v - 1].start + t[v - 1].block * (blocks + t[v - 1].extra) * (double)ceil_div(wgs, kCus) +
                        (sp > 1 ? 2 + (double)(sp * p->rows * p->n) * 2.4e-6 : 0);
      if (best == 0 || us < least) best = v, least = us;
    }
    if (best == 0) return GEMM_ERR_UNSUPPORTED;
    take(best);
  }
  s->splits = splits();
  s->ws = s->splits > 1 ? s->splits * p->rows * p->n * 4 : 0;
  return GEMM_OK;
}

}  // namespace

extern "C" {

gemm_status_t experts_sort_workspace_bytes(int64_t slots, int64_t experts, int64_t* out) {
  if (!out || slots < 0) return GEMM_ERR_INVALID;
  if (experts < 1 || experts > kMaxExperts || slots > kMax32) return GEMM_ERR_UNSUPPORTED;
  const SortShape s = sort_shape(slots);
  *out = s.blocks > 1 ? s.blocks * (experts + 1) * 4 : 0;
  return GEMM_OK;
}

gemm_status_t experts_sort(const void* ids, int id_bits, int64_t slots, int64_t experts, int32_t* offsets,
                           int32_t* order, int32_t* rows, void* workspace, int64_t workspace_bytes, void* stream) {
  int64_t need = 0;
  gemm_status_t st = experts_sort_workspace_bytes(slots, experts, &need);
  if (st != GEMM_OK) return st;
  if ((id_bits != 32 && id_bits != 64) || !offsets || (slots > 0 && (!ids || !order || !rows)) ||
      (need > 0 && (!workspace || workspace_bytes < need)))
    return GEMM_ERR_INVALID;
  int cu = 0;
  st = device_cus(&cu);
  if (st != GEMM_OK) return st;
  const SortShape s = sort_shape(slots);
  spt::SortArgs a;
  a.ids = ids;
  a.id64 = id_bits == 64;
  a.rows = (int)slots;
  a.experts = (int)experts;
  a.per_block = (int)s.per_block;
  a.blocks = (int)s.blocks;
  a.counts = (int*)workspace;
  a.offsets = offsets;
  a.slots = order;
  a.rows_of = rows;
  const int keys = (int)experts + 1;
  if (s.blocks == 1) return launch(spt::sort_one_fn(), dim3(1), 1024, (17 * keys + 16) * 4, &a, stream);
  st = launch(spt::sort_hist_fn(), dim3((unsigned)s.blocks), 1024, keys * 4, &a, stream);
  if (st != GEMM_OK) return st;
  return launch(spt::sort_place_fn(), dim3((unsigned)s.blocks), 1024, (18 * keys + 16) * 4, &a, stream);
}

gemm_status_t experts_gather(const void* x, gemm_dtype_t dtype, int64_t tokens, int64_t top_k, int64_t width,
                             int64_t ldx, const int32_t* rows, const int32_t* kept, void* out, int64_t ldo,
                             int zero_rest, void* stream) {
  gemm_status_t st = check_route(dtype, tokens, top_k, width);
  if (st != GEMM_OK) return st;
  if (ldx < width || ldo < width) return GEMM_ERR_INVALID;
  if (tokens == 0 || top_k == 0 || width == 0) return GEMM_OK;
  if (!x || !rows || !kept || !out) return GEMM_ERR_INVALID;
  spt::RouteArgs a{};
  dim3 grid;
  st = route_grid(tokens, width, &a.lanes_log2, &grid);
  if (st != GEMM_OK) return st;
  a.src = (const char*)x;
  a.dst = (char*)out;
  a.rows_of = rows;
  a.kept = kept;
  a.ld_src = ldx;
  a.ld_dst = ldo;
  a.tokens = (int)tokens;
  a.top_k = (int)top_k;
  a.width = (int)width;
  a.zero_rest = zero_rest != 0;
  return launch(spt::gather_fn((int)dtype), grid, 256, 0, &a, stream);
}

gemm_status_t experts_combine(const void* y, gemm_dtype_t dtype, int64_t tokens, int64_t top_k, int64_t width,
                              int64_t ldy, const int32_t* rows, const int32_t* kept, const void* weights,
                              gemm_dtype_t weight_dtype, void* out, int64_t ldo, void* stream) {
  gemm_status_t st = check_route(dtype, tokens, top_k, width);
  if (st != GEMM_OK) return st;
  if (ldy < width || ldo < width || (weights && !is_dtype(weight_dtype))) return GEMM_ERR_INVALID;
  if (tokens == 0 || width == 0) return GEMM_OK;
  if (!out || !kept || (top_k > 0 && (!y || !rows))) return GEMM_ERR_INVALID;
  spt::RouteArgs a{};
  dim3 grid;
  st = route_grid(tokens, width, &a.lanes_log2, &grid);
  if (st != GEMM_OK) return st;
  a.src = (const char*)y;
  a.dst = (char*)out;
  a.rows_of = rows;
  a.kept = kept;
  a.weights = weights;
  a.ld_src = ldy;
  a.ld_dst = ldo;
  a.tokens = (int)tokens;
  a.top_k = (int)top_k;
  a.width = (int)width;
  return launch(spt::combine_fn((int)dtype, weights ? (int)weight_dtype : 3), grid, 256, 0, &a, stream);
}

gemm_status_t experts_combine_grad(const void* dout, int64_t lddo, const void* y, gemm_dtype_t dtype, int64_t tokens,
                                   int64_t top_k, int64_t width, int64_t ldy, const int32_t* rows,
                                   const int32_t* kept, const void* weights, gemm_dtype_t weight_dtype, void* dy,
                                   int64_t lddy, void* dweights, int zero_rest, void* stream) {
  gemm_status_t st = check_route(dtype, tokens, top_k, width);
  if (st != GEMM_OK) return st;
  if (lddo < width || ldy < width || lddy < width || (weights && !is_dtype(weight_dtype))) return GEMM_ERR_INVALID;
  if (tokens == 0 || top_k == 0) return GEMM_OK;
  if (!rows || !kept || (width > 0 && (!dout || !y || !dy)) || (weights && !dweights)) return GEMM_ERR_INVALID;
  if (tokens * 256 > kMax32 || width > kMax32 - 2048) return GEMM_ERR_UNSUPPORTED;
  spt::RouteArgs a{};
  a.src = (const char*)y;
  a.dout = (const char*)dout;
  a.dst = (char*)dy;
  a.rows_of = rows;
  a.kept = kept;
  a.weights = weights;
  a.dweights = dweights;
  a.ld_src = ldy;
  a.ld_dst = lddy;
  a.ld_dout = lddo;
  a.tokens = (int)tokens;
  a.top_k = (int)top_k;
  a.width = (int)width;
  a.zero_rest = zero_rest != 0;
  return launch(spt::combine_grad_fn((int)dtype, weights ? (int)weight_dtype : 3), dim3((unsigned)tokens), 256, 0, &a,
                stream);
}

gemm_status_t gemm_grouped_workspace_bytes(const gemm_grouped_t* p, const void* X, const void* Y, int64_t* out) {
  GroupedShape s;
  if (!out) return GEMM_ERR_INVALID;
  const gemm_status_t st = grouped_shape(p, X, Y, &s);
  if (st == GEMM_OK) *out = s.ws;
  return st;
}

gemm_status_t gemm_grouped_run(const gemm_grouped_t* p, const void* X, const void* Y, void* out,
                               const int32_t* offsets, void* workspace, int64_t workspace_bytes, void* stream) {
  GroupedShape s;
  gemm_status_t st = grouped_shape(p, X, Y, &s);
  if (st != GEMM_OK) return st;
  const bool gb = p->mode == GEMM_GROUPED_GRAD_B, fwd = p->mode == GEMM_GROUPED_FORWARD;
  const int64_t out_n = fwd ? p->n : p->k;
  if (out_n == 0 || (gb ? p->experts == 0 || p->n == 0 : p->rows == 0)) return GEMM_OK;
  if (!out || !offsets) return GEMM_ERR_INVALID;
  // operands that hold at least one element have to be there
  if ((s.x.rows > 0 && s.x.cols > 0 && !X) || (s.y.rows > 0 && s.y.cols > 0 && !Y)) return GEMM_ERR_INVALID;
  if (s.ws > 0 && (!workspace || (uintptr_t)workspace % 16 != 0 || workspace_bytes < s.ws)) return GEMM_ERR_INVALID;

  const bool deep = s.tile == 32 && grouped_deep(p, Y);
  const spt::GroupedEntry entry = spt::grouped_entry((int)p->mode, s.tile, deep, p->in_dtype == GEMM_BF16,
                                                       s.splits > 1 ? (int)GEMM_F32 : (int)p->out_dtype);
  const int64_t tiles_m = ceil_div(p->n, entry.bm), tiles_n = ceil_div(out_n, entry.bn);
  const int64_t units = gb ? p->experts * tiles_m * tiles_n
                           : spt::max_row_blocks(p->rows, p->experts + 1, entry.bm) * tiles_n * s.splits;
  if (units > kMaxUnits) return GEMM_ERR_UNSUPPORTED;
  int cu = 0;
  st = device_cus(&cu);
  if (st != GEMM_OK) return st;
  const int64_t grid = units < (int64_t)cu * entry.per_cu ? units : (int64_t)cu * entry.per_cu;

  st = pad_operand(s.x, &X, (char*)workspace, stream);
  if (st != GEMM_OK) return st;
  st = pad_operand(s.y, &Y, (char*)workspace, stream);
  if (st != GEMM_OK) return st;

  spt::GroupedArgs a;
  a.X = (const char*)X;
  a.Y = (const char*)Y;
  a.C = (char*)out;
  a.offsets = offsets;
  a.rows = (int)p->rows;
  a.experts = (int)p->experts;
  a.m = (int)p->n;
  a.n = (int)out_n;
  a.kc = (int)(fwd ? p->k : p->n);
  a.ldx = s.x.ld;
  a.ldy = s.y.ld;
  a.ldc = p->ldo;
  a.sy = s.y.stride;
  a.sc = gb ? p->stride : 0;
  a.tiles_m = (int)tiles_m;
  a.tiles_n = (int)tiles_n;
  a.group_m = 8;
  a.grid = (int)grid;
  a.units = (int)units;
  a.rest = p->zero_rest != 0;
  // Short sums write as fast as HBM takes it, and non-temporal stores are taken faster (8190 rows, 16
  // experts, 4096 x 2048: fp32 258 -> 224 us, bf16 188 -> 159); among long ones they only leave the caches
  // (16384 rows, 8 experts, 8192 x 4096: 886 -> 917).
  a.nt = (gb ? ceil_div(p->rows, p->experts) : a.kc) < 1024;
  a.splits = (int)s.splits;
  a.plane = p->rows * out_n;
  if (s.splits == 1) return launch(entry.fn, dim3((unsigned)grid), entry.threads, 0, &a, stream);
  a.C = (char*)workspace + s.planes;
  a.ldc = out_n;
  st = launch(entry.fn, dim3((unsigned)grid), entry.threads, 0, &a, stream);
  if (st != GEMM_OK) return st;
  return add_planes((const float*)a.C, out, a.rest ? nullptr : offsets, p->experts, p->ldo, p->rows, out_n, s.splits,
                    (int)p->out_dtype, stream);
}

gemm_status_t gemm_w4_packed_bytes(int64_t matrices, int64_t n, int64_t k, int group, int has_zeros, int64_t* out) {
  if (!out || matrices < 0 || n < 0 || k < 0) return GEMM_ERR_INVALID;
  const int64_t lim = (int64_t)1 << 24;
  if ((group != 32 && group != 64 && group != 128) || n > lim || k > lim || matrices > kMaxGroups ||
      w4_too_large(matrices, n, k))
    return GEMM_ERR_UNSUPPORTED;
  *out = w4_blocks(matrices, n, k) * (1024 + 16 * (128 / group) * (has_zeros ? 3 : 2));
  return GEMM_OK;
}

gemm_status_t gemm_w4_pack(const uint8_t* q, const void* scales, const uint8_t* zeros, int64_t matrices, int64_t n,
                           int64_t k, int group, void* packed, void* stream) {
  int64_t bytes = 0;
  gemm_status_t st = gemm_w4_packed_bytes(matrices, n, k, group, zeros != nullptr, &bytes);
  if (st != GEMM_OK) return st;
  if (bytes == 0) return GEMM_OK;
  if (!q || !scales || !packed || (uintptr_t)packed % 16 != 0) return GEMM_ERR_INVALID;
  int cu = 0;
  st = device_cus(&cu);
  if (st != GEMM_OK) return st;
  spt::W4PackArgs a;
  a.q = q;
  a.scales = (const unsigned short*)scales;
  a.zeros = zeros;
  a.packed = (char*)packed;
  a.matrices = matrices;
  a.n = (int)n;
  a.k = (int)k;
  a.group = group;
  const int64_t blocks = w4_blocks(matrices, n, k);
  st = launch(spt::w4_pack_fn(), dim3(stream_grid(blocks * 256)), 256, 0, &a, stream);
  if (st != GEMM_OK) return st;
  return launch(spt::w4_pack_groups_fn(), dim3(stream_grid(blocks * 16 * (128 / group))), 256, 0, &a, stream);
}

gemm_status_t gemm_w4_workspace_bytes(const gemm_w4_t* p, int has_offsets, int64_t* out) {
  if (!out) return GEMM_ERR_INVALID;
  W4Shape s;
  const gemm_status_t st = w4_shape(p, has_offsets != 0, &s);
  if (st == GEMM_OK) *out = s.ws;
  return st;
}

gemm_status_t gemm_w4_run(const gemm_w4_t* p, const void* x, const void* packed, const int32_t* offsets, void* out,
                          void* workspace, int64_t workspace_bytes, void* stream) {
  W4Shape s;
  int cu = 0;
  gemm_status_t st = w4_shape(p, offsets != nullptr, &s);
  if (st != GEMM_OK) return st;
  if (p->rows == 0 || p->n == 0) return GEMM_OK;
  if (!out || (p->k > 0 && (!x || (p->matrices > 0 && (!packed || (uintptr_t)packed % 16 != 0))))) return GEMM_ERR_INVALID;
  if (s.ws > 0 && (!workspace || (uintptr_t)workspace % 4 != 0 || workspace_bytes < s.ws)) return GEMM_ERR_INVALID;
  st = device_cus(&cu);
  if (st != GEMM_OK) return st;
  const int gpk = 128 / p->group;
  const int64_t blocks = w4_blocks(p->matrices, p->n, p->k);
  spt::W4Args a;
  a.x = (const char*)x;
  a.w = (const char*)packed;
  a.scales = a.w + blocks * 1024;
  a.zeros = a.scales + blocks * 16 * gpk * 2;
  a.out = s.splits > 1 ? (char*)workspace : (char*)out;
  a.offsets = offsets;
  a.ldx = p->ldx;
  a.ldo = p->ldo;
  a.plane = p->rows * p->n;
  a.rows = (int)p->rows;
  a.experts = (int)p->matrices;
  a.n = (int)p->n;
  a.k = (int)p->k;
  a.n16 = (int)ceil_div(p->n, 16);
  a.kb = (int)ceil_div(p->k, 128);
  a.splits = (int)s.splits;
  a.rest = p->zero_rest != 0;
  a.out_dtype = (int)p->out_dtype;
  st = launch(s.entry.fn, dim3((unsigned)(s.nblocks * s.splits), (unsigned)s.grid_y), 64 * s.entry.waves, 0, &a,
              stream);
  if (st != GEMM_OK || s.splits == 1) return st;
  return add_planes((const float*)workspace, out, a.rest ? nullptr : offsets, p->matrices, p->ldo, p->rows, p->n, s.splits,
                    a.out_dtype, stream);
}

}  // extern "C"
