// Shared definitions of the microscaled operators and the norm: kernel arguments, the layout, conversions.
#pragma once

#include "spt_common.h"

namespace spt {

// ------------------------------------------------------------------------------ layout
constexpr int kMxBlock = 32;      // values that share a scale
constexpr int kMxScaleRows = 64;  // rows whose scales of one block lie together
constexpr int kMxUnitRows = 16;  // rows that a workgroup of the streams takes

SPT_HD int64_t mx_blocks(int64_t k) { return (k + 127) / 128 * 4; }  // of a row, with those behind k
SPT_HD int64_t mx_row_bytes(int64_t k, int bits) { return mx_blocks(k) * (4 * bits); }
SPT_HD int64_t mx_scale_at(int64_t row, int64_t block, int64_t blocks) {
  return ((row / kMxScaleRows) * blocks + block) * kMxScaleRows + row % kMxScaleRows;
}

// ------------------------------------------------------------------------------ arguments
struct MxQuantArgs {
  const char* x;
  unsigned char* codes;
  unsigned char* scales;
  int64_t rows, ldx;
  int k, blocks;        // blocks of a row
  int64_t units;        // of 16 rows by 512 columns
};
struct MxValuesArgs {
  const unsigned char* codes;
  const unsigned char* scales;
  char* out;
  int64_t rows, ldo;
  int k, blocks;
  int64_t units;
};
struct MxPackArgs {
  const unsigned char* codes;
  const unsigned char* scales;
  unsigned char* out_codes;
  unsigned char* out_scales;
  int64_t rows, ldc, lds;
  int k, blocks;
  int64_t units;
};

struct MxGemmArgs {
  const char* a;
  const char* as;
  const char* b;
  const char* bs;
  char* c;              // output, or fp32 planes of a cut sum
  int m, n;
  int blocks;           // scale blocks of a row
  int ksteps;           // 128 values of k each
  int64_t ldc;
  int out_dtype;
  int tiles_m, tiles_n;
  int group_m;
  int units;            // output tiles times parts of the sum
  int splits;
  int per;              // K-tiles of one part (the skinny kernel has one)
  int64_t plane;        // elements between planes
  int grid;
  int nt;               // non-temporal stores
};

struct NormArgs {
  const char* x;
  const char* r;        // residual, or null
  const char* w;        // weight, or null
  char* h;
  char* y;              // y, or codes
  unsigned char* scales;
  int64_t rows, ldx, ldr, ldh, ldy;
  int n, blocks, wtype;
  float eps;
  int64_t per;          // rows of a workgroup
  int lanes;
};
struct NormGradArgs {
  const char* dy;
  const char* h;
  const char* w;
  const char* dh;       // or null
  char* dx;
  float* parts;         // [workgroups][n] sums of dweight, or null
  int64_t rows, lddy, ldh, lddh, lddx;
  int n, wtype;
  float eps;
  int64_t per;
  int lanes;
};
struct NormPartsArgs {
  const float* parts;
  char* out;
  int n, count, wtype;
};

const void* mx_quantize_fn(int dtype, int bits);
const void* mx_values_fn(int dtype, int bits);
const void* mx_pack_fn(int bits);
// out: 0 the input's type, else bits; c: pieces of eight values to a thread (1, 2, and the 16-bit norms 4; up to 1024 threads), -1:
// rows of `lanes` threads of 256, 0: rows of any length, 512 threads, -2: gradients with 32 bytes of LDS to a piece, 1024 threads, -3:
// gradients with rows of `lanes` threads, whole waves, side by side
const void* norm_fn(int dtype, int out, int c);
const void* norm_grad_fn(int dtype, int c);
const void* norm_parts_fn();

struct MxEntry {
  const void* fn;
  int bm, bn, threads, ksteps;  // k-steps of a K-tile
};
// fa, fb: bits; exact: products through bf16
MxEntry mx_tile_entry(int fa, int fb, bool exact, int bm);  // bm: 32, 64, 128
// out: 0 f16, 1 bf16, 2 f32
MxEntry mx_pp_entry(int fa, int fb, int out);
MxEntry mx_skinny_entry(int fa, int fb, bool exact, int mt);  // mt: blocks of 16 rows (1, 2)

}  // namespace spt
