// Host side of include/microscale.h: argument checks, the choice of a kernel, launches. Nothing here allocates or
// synchronises, and no state outlives a call but the devices' properties.
#include <cmath>

#include "microscale.h"
#include "spt_host.h"
#include "spt_mx.h"

namespace {

using namespace spt;

constexpr int64_t kMaxRows = kMax32 - 63;             // their number rounded up to 64 stays inside 32 bits
constexpr int64_t kMaxK = (int64_t)1 << 22;           // 256 rows of it stay inside a buffer's 32-bit offsets
constexpr int64_t kMaxNorm = (int64_t)1 << 24;
constexpr int64_t kMaxLdc = (int64_t)1 << 20;
constexpr int64_t kMaxTiles = (int64_t)1 << 24;       // of 32 x 64, the smallest tile's half

bool on16(const void* p) { return (uintptr_t)p % 16 == 0; }

gemm_status_t check_mx(int64_t rows, int64_t k, int bits) {
  if (rows < 0 || k < 0 || (bits != 4 && bits != 8)) return GEMM_ERR_INVALID;
  if (rows > kMaxRows || k > kMaxK) return GEMM_ERR_UNSUPPORTED;
  return GEMM_OK;
}

// Units of 16 rows by 512 columns, and the workgroups that walk over them. The last 64 rows have all theirs: rows behind the last
// one have scales, zeros.
struct Units {
  int64_t units;
  unsigned grid;
};
Units mx_units(int64_t rows, int64_t blocks) {
  Units u;
  u.units = round_up(rows, kMxScaleRows) / kMxUnitRows * ceil_div(blocks, 16);
  u.grid = (unsigned)(u.units < 65536 ? u.units : 65536);
  return u;
}

// ---------------------------------------------------------------------------------- products
enum MxKernel { kSkinny16, kSkinny32, kTile32, kTile64, kTile128, kTwoGroup, kMxKernels };

struct MxShape {
  MxKernel kernel;
  MxEntry entry;
  bool exact;
  int64_t tiles_m, tiles_n, splits, per, ws;  // per: K-tiles of one part of a sum
};

MxEntry mx_entry(MxKernel kernel, const gemm_mx_t* p, bool exact, bool planes) {
  const int fa = p->a_bits, fb = p->b_bits;
  switch (kernel) {
    case kSkinny16: return mx_skinny_entry(fa, fb, exact, 1);
    case kSkinny32: return mx_skinny_entry(fa, fb, exact, 2);
    case kTile32: return mx_tile_entry(fa, fb, exact, 32);
    case kTile64: return mx_tile_entry(fa, fb, exact, 64);
    case kTile128: return mx_tile_entry(fa, fb, exact, 128);
    default: return mx_pp_entry(fa, fb, planes ? (int)GEMM_F32 : (int)p->out_dtype);
  }
}

// The kernel and the parts of a sum: the least time by this model, in us. A start; the longer of the workgroups' rounds over the
// compute units (k-steps times what one takes, and the tile's own start and end) and the bytes; and, with parts, the second pass
// over their planes. Tiles run two to a compute unit, and a workgroup alone on its own takes its k-steps faster. A workgroup draws only
// so many bytes at once, so that fewer than 170 tiles do not fill the memory (1 x 8192 x 8192, 8 x 8: 16.9 us in four parts of 64 tiles,
// 23.6 in two). The constants are a fit to 3400 measured shapes (1 .. 16384 rows, N 64 .. 28672, K 100 .. 14336); on 1800 of them the choice
// takes 2.3 % longer than the best kernel of each shape, 82 % at worst (1386 x 11469 x 650, 4 x 4 in fp32: 34 us against 18), where rules on
// the numbers of rows and tiles took 25 %. On 2000 other shapes of the same ranges it takes 3.6 % longer, more than 10 % on 268 of them, 58 %
// at worst (2442 x 5248 x 192, 4 x 4: 15.6 us against 9.9 with two groups); the worst have sums of 100 to 700. Where power holds the
// matrix cores back its times are too short (8192^3 8 x 8: 275 us, 364 measured), for all kernels alike.
void mx_choose(const gemm_mx_t* p, MxShape* s) {
  // by format: 4 x 4, 8 x 4, 8 x 8, and the last two exact
  struct Cost {
    double start, solo[5], pair[5], tile[3], out;
  };
  static const Cost costs[kMxKernels] = {
      {2.8, {.60, .60, 1.05, .63, 1.14}, {}, {}, .3},
      {2.4, {.90, 1.35, 1.56, .98, 1.60}, {}, {}, .3},
      {3.0, {.20, .235, .306, .485, .56}, {.385, .54, .59, .80, .915}, {}, .45},
      {3.7, {.22, .34, .42, .665, .72}, {.405, .565, .65, 1.0, 1.11}, {}, .4},
      {5.0, {.345, .50, .63, .97, 1.07}, {.50, .725, .90, 1.46, 1.70}, {}, .35},
      {5.0, {}, {.66, .90, .98}, {3.2, 3.3, 4.8}, .24}};
  static const int parts[] = {1, 2, 3, 4, 6, 8, 12, 16};
  const int f = (p->a_bits == 4 ? 0 : p->b_bits == 4 ? 1 : 2) + (s->exact ? 2 : 0);
  const int64_t ksteps = mx_blocks(p->k) / 4;
  const double operands = ((double)p->n * p->b_bits + (double)p->m * p->a_bits) * (double)p->k / 8e6;
  const double plane = (double)p->m * (double)p->n * 4e-6;
  double least = 0;
  bool any = false;
  for (int i = 0; i < kMxKernels; ++i) {
    const MxKernel kernel = (MxKernel)i;
    const bool skinny = kernel <= kSkinny32, pp = kernel == kTwoGroup;
    // a workgroup of the skinny kernel has all rows, and as many columns as keep it the only one on its compute unit
    if (skinny && (p->m > (kernel == kSkinny16 ? 16 : 32) || p->n > 16 * kCus)) continue;
    if (pp && s->exact) continue;
    const MxEntry e = mx_entry(kernel, p, s->exact, false);
    const Cost& c = costs[i];
    const int64_t tm = ceil_div(p->m, e.bm), tn = ceil_div(p->n, e.bn), kt = ceil_div(ksteps, e.ksteps);
    for (int sp : parts) {
      const int64_t units = tm * tn * sp, per = ceil_div(kt, sp);
      if (sp > 1 && (skinny || units > 4 * kCus || kt < 2 * sp)) break;
      if (pp && (kt < 2 || kt - (kt - 1) / per * per < 2)) continue;  // its pipeline has at least two K-tiles, those of the last part too
      double work;
      if (skinny) work = c.solo[f] * (double)ceil_div(ksteps, 8);
      else if (pp) work = (double)ceil_div(units, kCus) * (c.pair[f] * (double)(per * e.ksteps) + c.tile[f]);
      else work = (units <= kCus ? c.solo[f] : (double)ceil_div(units, 2 * kCus) * c.pair[f]) * (double)(per * e.ksteps);
      const double out = sp > 1 ? plane * sp : plane * (p->out_dtype == GEMM_F32 ? 1 : .5);
      const double drawn = skinny ? .2 : pp || units > 166 ? .18 : 30. / (double)units;  // us for a megabyte
      const double bytes = drawn * operands + c.out * out;
      const double us = c.start + (work > bytes ? work : bytes) + (sp > 1 ? 2.7 + .4 * out : 0);
      if (any && us >= least) continue;
      any = true;
      least = us;
      s->kernel = kernel;
      s->splits = kt > 0 ? ceil_div(kt, per) : 1;
      s->per = per;
    }
  }
}

gemm_status_t mx_shape(const gemm_mx_t* p, MxShape* s) {
  if (!p || !is_dtype(p->out_dtype) || p->ldc < p->n) return GEMM_ERR_INVALID;
  gemm_status_t st = check_mx(p->m, p->k, p->a_bits);
  if (st == GEMM_OK) st = check_mx(p->n, p->k, p->b_bits);
  if (st != GEMM_OK) return st;
  if ((p->a_bits == 4 && p->b_bits == 8) || p->ldc >= kMaxLdc) return GEMM_ERR_UNSUPPORTED;
  if (ceil_div(p->m, 32) * ceil_div(p->n, 64) > kMaxTiles) return GEMM_ERR_UNSUPPORTED;
  s->exact = p->out_dtype == GEMM_F32 && p->a_bits == 8;
  s->kernel = kTile32;
  s->splits = 1;
  s->per = 0;
  mx_choose(p, s);
  s->entry = mx_entry(s->kernel, p, s->exact, s->splits > 1);
  s->tiles_m = ceil_div(p->m, s->entry.bm);
  s->tiles_n = ceil_div(p->n, s->entry.bn);
  s->ws = s->splits > 1 ? s->splits * p->m * p->n * 4 : 0;
  return GEMM_OK;
}

// ---------------------------------------------------------------------------------- norm
// Pieces of eight values a thread keeps (0: a row too long for registers; -1: a row is a part of a wave's; -2: gradients of
// long rows with dweight's sums in LDS; -3: gradients of rows side by side), threads of a row and of a workgroup, bytes of LDS, rows of a workgroup.
constexpr int64_t kGradLdsPieces = 4992;  // 156 KB of the 160
struct NormShape {
  int c, lanes, threads, lds;
  int64_t per, grid;
};
// Figures here: the same operands again and again. A thread has as few pieces as 1024 threads allow (with the residual: 300 rows of 4096 bf16 4.0 us, 4.3 with two pieces to half the
// threads; 1003 rows of 4097 fp32 12.8, 14.1), and a workgroup neighbouring rows, so that all workgroups are on the compute units at once
// (6 waves to a SIMD, for the gradients' registers 5: 8192 rows of 4096 bf16 60 us, 65 with 6).
NormShape norm_shape(int64_t rows, int64_t n, gemm_dtype_t dtype, bool mx, bool grad) {
  NormShape s{};
  const int64_t pieces = mx ? mx_blocks(n) * (kMxBlock / 8) : ceil_div(n, 8);
  int64_t per_cu;
  if (pieces <= 64) {
    s.c = -1;
    s.threads = 256;
    for (s.lanes = mx ? 16 : 4; s.lanes < pieces;) s.lanes *= 2;
    per_cu = grad ? 3 : 6;
  } else {
    if (pieces <= 1024) s.c = 1;
    else if (pieces <= 2048) s.c = 2;
    else if (grad) s.c = pieces <= kGradLdsPieces ? -2 : 0;
    else s.c = pieces <= 4096 && dtype != GEMM_F32 ? 4 : 0;
    s.threads = s.c > 0 ? (int)round_up(ceil_div(pieces, s.c), 64) : s.c < 0 ? 1024 : 512;
    if (s.c == -2) s.lds = (int)pieces * 32;
    s.lanes = s.threads;
    // Gradients of few rows side by side, where one after the other leaves the compute units few waves: 2048 rows of 2560 bf16 16.6 us
    // (21.0), 16384 of 1024 36.9 (41.5); but 8192 of 2048 38 (34), 4096 of 4096 37 (33), 65536 of 600 114 (87).
    if (grad && s.c == 1 && s.lanes < 512 && rows * s.lanes <= (s.lanes == 128 ? 2 : 1) << 20) {
      s.c = -3;
      s.threads = 1024 / s.lanes * s.lanes;
    }
    per_cu = (grad ? 1280 : 1536) / s.threads;
  }
  const int64_t together = s.threads / s.lanes;  // rows of a workgroup at once
  const int64_t fit = kCus * per_cu;
  s.per = ceil_div(rows, fit);
  // every workgroup leaves a plane of dweight: at least eight rows to one, as long as all compute units have one
  if (grad && s.per < 8) s.per = ceil_div(rows, kCus) < 8 ? ceil_div(rows, kCus) : 8;
  s.per = round_up(s.per, together);
  s.grid = s.per > 0 ? ceil_div(rows, s.per) : 0;
  return s;
}

gemm_status_t check_norm(const norm_rms_t* p) {
  if (!p || p->rows < 0 || p->n < 0 || !is_dtype(p->dtype) || !is_dtype(p->weight_dtype)) return GEMM_ERR_INVALID;
  if (!(p->eps >= 0.f) || !std::isfinite(p->eps)) return GEMM_ERR_INVALID;
  if (p->rows > kMaxRows || p->n > kMaxNorm) return GEMM_ERR_UNSUPPORTED;
  return GEMM_OK;
}

// Whether rows of two results share memory: exact for one row and for rows of one stride; of two strides only a common first address.
bool rows_meet(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t rows, int64_t row_bytes, int es) {
  const __int128 d = a < b ? (const char*)b - (const char*)a : (const char*)a - (const char*)b;
  if (d == 0 || rows == 1 || lda != ldb) return d == 0 || (rows == 1 && d < row_bytes);
  const __int128 step = (__int128)lda * es;
  if (d >= step * rows) return false;
  const int64_t before = (int64_t)(d / step), rest = (int64_t)(d - before * step);  // the lower one's last row that begins ahead of the upper one
  return rest < row_bytes || (before + 1 < rows && step - rest < row_bytes);
}

gemm_status_t run_norm(const norm_rms_t* p, int out, const void* x, const void* residual, const void* weight, void* h,
                       void* y, void* scales, void* stream) {
  gemm_status_t st = check_norm(p);
  if (st != GEMM_OK) return st;
  if (out && p->n > kMaxK) return GEMM_ERR_UNSUPPORTED;
  if (p->ldx < p->n || (residual && (p->ldr < p->n || p->ldh < p->n)) || (!out && p->ldy < p->n)) return GEMM_ERR_INVALID;
  if (p->rows == 0 || p->n == 0) return GEMM_OK;
  if (!x || !y || (residual && !h) || (out && (!scales || !on16(y) || !on16(scales)))) return GEMM_ERR_INVALID;
  if (residual) {  // x's memory may take h or y, but not both
    const int es = p->dtype == GEMM_F32 ? 4 : 2;
    if (out ? y == h || scales == h : rows_meet(y, p->ldy, h, p->ldh, p->rows, p->n * es, es)) return GEMM_ERR_INVALID;
  }
  int cu = 0;
  st = device_cus(&cu);
  if (st != GEMM_OK) return st;
  NormArgs a{};
  a.x = (const char*)x;
  a.r = (const char*)residual;
  a.w = (const char*)weight;
  a.h = (char*)h;
  a.y = (char*)y;
  a.scales = (unsigned char*)scales;
  a.rows = p->rows; a.ldx = p->ldx; a.ldr = p->ldr; a.ldh = p->ldh; a.ldy = p->ldy;
  a.n = (int)p->n;
  a.blocks = (int)mx_blocks(p->n);
  a.wtype = (int)p->weight_dtype;
  a.eps = p->eps;
  const NormShape s = norm_shape(p->rows, p->n, p->dtype, out != 0, false);
  a.per = s.per;
  a.lanes = s.lanes;
  return launch(norm_fn((int)p->dtype, out, s.c), dim3((unsigned)s.grid), s.threads, 0, &a, stream);
}

gemm_status_t check_grad(const norm_rms_grad_t* p) {
  if (!p) return GEMM_ERR_INVALID;
  norm_rms_t f{};
  f.rows = p->rows; f.n = p->n; f.dtype = p->dtype; f.weight_dtype = p->weight_dtype; f.eps = p->eps;
  return check_norm(&f);
}
NormShape grad_shape(const norm_rms_grad_t* p) { return norm_shape(p->rows, p->n, p->dtype, false, true); }

}  // namespace

extern "C" {

gemm_status_t mx_bytes(int64_t rows, int64_t k, int bits, int64_t* codes, int64_t* scales) {
  if (!codes || !scales) return GEMM_ERR_INVALID;
  const gemm_status_t st = check_mx(rows, k, bits);
  if (st != GEMM_OK) return st;
  *codes = rows * mx_row_bytes(k, bits);
  *scales = round_up(rows, kMxScaleRows) * mx_blocks(k);
  return GEMM_OK;
}

gemm_status_t mx_quantize(const void* x, gemm_dtype_t dtype, int64_t rows, int64_t k, int64_t ldx, int bits, void* codes,
                          void* scales, void* stream) {
  gemm_status_t st = check_mx(rows, k, bits);
  if (st != GEMM_OK) return st;
  if (!is_dtype(dtype) || ldx < k) return GEMM_ERR_INVALID;
  if (rows == 0 || k == 0) return GEMM_OK;
  if (!x || !codes || !scales || !on16(codes) || !on16(scales)) return GEMM_ERR_INVALID;
  int cu = 0;
  st = device_cus(&cu);
  if (st != GEMM_OK) return st;
  MxQuantArgs a;
  a.x = (const char*)x;
  a.codes = (unsigned char*)codes;
  a.scales = (unsigned char*)scales;
  a.rows = rows; a.ldx = ldx;
  a.k = (int)k;
  a.blocks = (int)mx_blocks(k);
  const Units u = mx_units(rows, a.blocks);
  a.units = u.units;
  return launch(mx_quantize_fn((int)dtype, bits), dim3(u.grid), 256, 0, &a, stream);
}

gemm_status_t mx_dequantize(const void* codes, const void* scales, int bits, int64_t rows, int64_t k, void* out,
                            gemm_dtype_t dtype, int64_t ldo, void* stream) {
  gemm_status_t st = check_mx(rows, k, bits);
  if (st != GEMM_OK) return st;
  if (!is_dtype(dtype) || ldo < k) return GEMM_ERR_INVALID;
  if (rows == 0 || k == 0) return GEMM_OK;
  if (!out || !codes || !scales || !on16(codes) || !on16(scales)) return GEMM_ERR_INVALID;
  int cu = 0;
  st = device_cus(&cu);
  if (st != GEMM_OK) return st;
  MxValuesArgs a;
  a.codes = (const unsigned char*)codes;
  a.scales = (const unsigned char*)scales;
  a.out = (char*)out;
  a.rows = rows; a.ldo = ldo;
  a.k = (int)k;
  a.blocks = (int)mx_blocks(k);
  const Units u = mx_units(rows, a.blocks);
  a.units = u.units;
  return launch(mx_values_fn((int)dtype, bits), dim3(u.grid), 256, 0, &a, stream);
}

gemm_status_t mx_pack(const void* codes, int64_t ldc, const void* scales, int64_t lds, int bits, int64_t rows, int64_t k,
                      void* out_codes, void* out_scales, void* stream) {
  gemm_status_t st = check_mx(rows, k, bits);
  if (st != GEMM_OK) return st;
  if (ldc < ceil_div(k * bits, 8) || lds < ceil_div(k, kMxBlock)) return GEMM_ERR_INVALID;
  if (rows == 0 || k == 0) return GEMM_OK;
  if (!codes || !scales || !out_codes || !out_scales || !on16(out_codes) || !on16(out_scales)) return GEMM_ERR_INVALID;
  int cu = 0;
  st = device_cus(&cu);
  if (st != GEMM_OK) return st;
  MxPackArgs a;
  a.codes = (const unsigned char*)codes;
  a.scales = (const unsigned char*)scales;
  a.out_codes = (unsigned char*)out_codes;
  a.out_scales = (unsigned char*)out_scales;
  a.rows = rows; a.ldc = ldc; a.lds = lds;
  a.k = (int)k;
  a.blocks = (int)mx_blocks(k);
  const Units u = mx_units(rows, a.blocks);
  a.units = u.units;
  return launch(mx_pack_fn(bits), dim3(u.grid), 256, 0, &a, stream);
}

gemm_status_t gemm_mx_workspace_bytes(const gemm_mx_t* p, int64_t* out) {
  if (!out) return GEMM_ERR_INVALID;
  MxShape s;
  const gemm_status_t st = mx_shape(p, &s);
  if (st == GEMM_OK) *out = s.ws;
  return st;
}

gemm_status_t gemm_mx_describe(const gemm_mx_t* p, gemm_mx_config_t* out) {
  if (!out) return GEMM_ERR_INVALID;
  MxShape s;
  const gemm_status_t st = mx_shape(p, &s);
  if (st != GEMM_OK) return st;
  out->kernel = s.kernel <= kSkinny32 ? 0 : s.kernel == kTwoGroup ? 2 : 1;
  out->bm = s.entry.bm;
  out->bn = s.entry.bn;
  out->splits = (int)s.splits;
  out->k_per_part = s.per * s.entry.ksteps * 128;
  out->through_bf16 = s.exact;
  return GEMM_OK;
}

gemm_status_t gemm_mx_run(const gemm_mx_t* p, const void* a_codes, const void* a_scales, const void* b_codes,
                          const void* b_scales, void* C, void* workspace, int64_t workspace_bytes, void* stream) {
  MxShape s;
  gemm_status_t st = mx_shape(p, &s);
  if (st != GEMM_OK) return st;
  if (p->m == 0 || p->n == 0) return GEMM_OK;
  if (!C || (p->k > 0 && (!a_codes || !a_scales || !b_codes || !b_scales))) return GEMM_ERR_INVALID;
  if (!on16(a_codes) || !on16(a_scales) || !on16(b_codes) || !on16(b_scales)) return GEMM_ERR_INVALID;
  if (s.ws > 0 && (!workspace || !on16(workspace) || workspace_bytes < s.ws)) return GEMM_ERR_INVALID;
  int cu = 0;
  st = device_cus(&cu);
  if (st != GEMM_OK) return st;
  MxGemmArgs a{};
  a.a = (const char*)a_codes;
  a.as = (const char*)a_scales;
  a.b = (const char*)b_codes;
  a.bs = (const char*)b_scales;
  a.c = s.splits > 1 ? (char*)workspace : (char*)C;
  a.m = (int)p->m;
  a.n = (int)p->n;
  a.blocks = (int)mx_blocks(p->k);
  a.ksteps = a.blocks / 4;
  a.ldc = s.splits > 1 ? p->n : p->ldc;
  a.out_dtype = s.splits > 1 ? (int)GEMM_F32 : (int)p->out_dtype;
  a.tiles_m = (int)s.tiles_m;
  a.tiles_n = (int)s.tiles_n;
  a.group_m = 8;
  a.splits = (int)s.splits;
  a.per = (int)s.per;
  a.plane = s.splits > 1 ? p->m * p->n : 0;
  a.units = (int)(s.tiles_m * s.tiles_n * s.splits);
  a.grid = s.kernel == kTwoGroup && a.units > cu ? cu : a.units;  // it walks over its tiles
  // 16-bit stores write whole lines, and past the caches they are taken faster; fp32 ones are not (2236 x 24448 x 448: 115 us, 63)
  a.nt = s.splits == 1 && p->out_dtype != GEMM_F32;
  st = launch(s.entry.fn, dim3((unsigned)a.grid), s.entry.threads, 0, &a, stream);
  if (st != GEMM_OK || s.splits == 1) return st;
  return add_planes((const float*)workspace, C, nullptr, 0, p->ldc, p->m, p->n, s.splits, (int)p->out_dtype, stream);
}

gemm_status_t norm_rms_run(const norm_rms_t* p, const void* x, const void* residual, const void* weight, void* h, void* y,
                           void* stream) {
  return run_norm(p, 0, x, residual, weight, h, y, nullptr, stream);
}

gemm_status_t norm_rms_mx_run(const norm_rms_t* p, int bits, const void* x, const void* residual, const void* weight,
                              void* h, void* codes, void* scales, void* stream) {
  if (bits != 4 && bits != 8) return GEMM_ERR_INVALID;
  return run_norm(p, bits, x, residual, weight, h, codes, scales, stream);
}

gemm_status_t norm_rms_grad_workspace_bytes(const norm_rms_grad_t* p, int wants_dweight, int64_t* out) {
  if (!out) return GEMM_ERR_INVALID;
  const gemm_status_t st = check_grad(p);
  if (st == GEMM_OK) *out = wants_dweight ? grad_shape(p).grid * p->n * 4 : 0;
  return st;
}

gemm_status_t norm_rms_grad_run(const norm_rms_grad_t* p, const void* dy, const void* h, const void* weight, const void* dh,
                                void* dx, void* dweight, void* workspace, int64_t workspace_bytes, void* stream) {
  gemm_status_t st = check_grad(p);
  if (st != GEMM_OK) return st;
  if (p->lddy < p->n || p->ldh < p->n || (dh && p->lddh < p->n) || (dx && p->lddx < p->n)) return GEMM_ERR_INVALID;
  if (p->n == 0 || (!dx && !dweight)) return GEMM_OK;
  if (p->rows > 0 && (!dy || !h)) return GEMM_ERR_INVALID;
  const NormShape s = grad_shape(p);
  const int64_t need = dweight ? s.grid * p->n * 4 : 0;
  if (need > 0 && (!workspace || !on16(workspace) || workspace_bytes < need)) return GEMM_ERR_INVALID;
  int cu = 0;
  st = device_cus(&cu);
  if (st != GEMM_OK) return st;
  if (p->rows > 0) {
    NormGradArgs a{};
    a.dy = (const char*)dy;
    a.h = (const char*)h;
    a.w = (const char*)weight;
    a.dh = (const char*)dh;
    a.dx = (char*)dx;
    a.parts = dweight ? (float*)workspace : nullptr;
    a.rows = p->rows; a.lddy = p->lddy; a.ldh = p->ldh; a.lddh = p->lddh; a.lddx = p->lddx;
    a.n = (int)p->n;
    a.wtype = (int)p->weight_dtype;
    a.eps = p->eps;
    a.per = s.per;
    a.lanes = s.lanes;
    st = launch(norm_grad_fn((int)p->dtype, s.c), dim3((unsigned)s.grid), s.threads, s.lds, &a, stream);
    if (st != GEMM_OK || !dweight) return st;
  }
  if (!dweight) return GEMM_OK;
  NormPartsArgs r;
  r.parts = (const float*)workspace;
  r.out = (char*)dweight;
  r.n = (int)p->n;
  r.count = (int)s.grid;  // no rows: zeros
  r.wtype = (int)p->weight_dtype;
  return launch(norm_parts_fn(), dim3((unsigned)ceil_div(p->n, 16)), 256, 0, &r, stream);
}

}  // extern "C"
