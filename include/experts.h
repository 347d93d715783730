/*
 * experts.h — C ABI of the experts' operators beside the dense products of gemm.h, for AMD Instinct
 * MI355X (gfx950): tokens sorted by expert and back, the experts' products over the sorted rows with
 * their gradients, and products with 4-bit weights.
 *
 * Rows sorted by expert. With E experts, `offsets` is E + 1 ascending 32-bit integers in device
 * memory: expert e owns rows [offsets[e], offsets[e + 1]). Rows from offsets[E] on belong to nobody, and
 * so do those before offsets[0], which is 0 where experts_sort made it: offsets + lo with the weights of
 * experts lo .. hi - 1 and E = hi - lo are the products of those experts alone. Kernels clamp what they
 * read from `offsets` (and from `rows`, the position of each slot) to the operands and their work to what
 * ascending offsets can make, so wrong contents give wrong results but no access out of range.
 *
 * Conventions of gemm.h hold: entry points only enqueue kernels on `stream` for the current device,
 * allocate nothing, never synchronise, return a gemm_status_t and throw nothing. Workspaces are the
 * caller's: a *_workspace_bytes function gives the size (0: none needed, NULL allowed), its contents
 * need no preparation, and calls that may overlap need one each. Outputs and workspaces must not
 * overlap an operand. All entry points may be recorded into a HIP graph (no memset nodes, only kernels),
 * after one call on that device outside the capture.
 * Dimensions are counted in elements, leading dimensions too.
 */
#ifndef SPT_EXPERTS_H
#define SPT_EXPERTS_H

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ tokens sorted by expert */

/*
 * Stable sort of `slots` expert ids (slot = token * top_k + j; 32- or 64-bit integers). An id outside
 * [0, experts) is dropped: it sorts behind the last expert.
 *   offsets [experts + 1]   as above; offsets[experts] is the number of kept slots
 *   order   [slots]         sorted position -> slot
 *   rows    [slots]         slot -> sorted position, a permutation; the slot is kept exactly when its
 *                           position is below offsets[experts]
 * One kernel up to 4096 slots, two beyond (the workspace holds the workgroups' counts).
 * Errors: GEMM_ERR_INVALID (sizes negative, a null pointer, id_bits not 32 or 64, workspace missing),
 *         GEMM_ERR_UNSUPPORTED (experts not in 1 .. 1024, slots beyond 2^31 - 1), GEMM_ERR_HIP.
 */
gemm_status_t experts_sort_workspace_bytes(int64_t slots, int64_t experts, int64_t* out);
gemm_status_t experts_sort(const void* ids, int id_bits, int64_t slots, int64_t experts, int32_t* offsets,
                           int32_t* order, int32_t* rows, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * out[rows[t * top_k + j]] = x[t] for every kept slot; `kept` points to offsets[experts].
 * Rows of `out` ([tokens * top_k], ldo) at dropped positions become zeros with zero_rest != 0 and
 * are left as they were otherwise. dtype F16, BF16 or F32; any element alignment.
 * Errors: GEMM_ERR_INVALID, GEMM_ERR_UNSUPPORTED (tokens * top_k beyond 2^31 - 1, a grid beyond HIP's
 *         limits), GEMM_ERR_HIP.
 */
gemm_status_t experts_gather(const void* x, gemm_dtype_t dtype, int64_t tokens, int64_t top_k, int64_t width,
                             int64_t ldx, const int32_t* rows, const int32_t* kept, void* out, int64_t ldo,
                             int zero_rest, void* stream);

/*
 * out[t] = sum over j = 0, 1, .. of weights[t * top_k + j] * y[rows[t * top_k + j]] over kept slots, in
 * fp32, rounded once to `dtype`; a token without kept slots gets zeros. weights NULL: ones (this is
 * experts_gather's gradient); weight_dtype F16, BF16 or F32.
 */
gemm_status_t experts_combine(const void* y, gemm_dtype_t dtype, int64_t tokens, int64_t top_k, int64_t width,
                              int64_t ldy, const int32_t* rows, const int32_t* kept, const void* weights,
                              gemm_dtype_t weight_dtype, void* out, int64_t ldo, void* stream);

/*
 * Gradients of experts_combine: dy[rows[s]] = weights[s] * dout[t] and, where weights are given,
 * dweights[s] = <dout[t], y[rows[s]]> (fp32 sums; the weights' type) for every kept slot s of token
 * t. A dropped slot has dweights 0 and its row of dy is zeros (zero_rest != 0) or left as it was.
 * Errors: as experts_gather; GEMM_ERR_UNSUPPORTED from 2^23 tokens on.
 */
gemm_status_t experts_combine_grad(const void* dout, int64_t lddo, const void* y, gemm_dtype_t dtype, int64_t tokens,
                                   int64_t top_k, int64_t width, int64_t ldy, const int32_t* rows,
                                   const int32_t* kept, const void* weights, gemm_dtype_t weight_dtype, void* dy,
                                   int64_t lddy, void* dweights, int zero_rest, void* stream);

/* ------------------------------------------------------------------ the experts' products */

typedef enum {
  GEMM_GROUPED_FORWARD = 0, /* C[i] = A[i] . B[e]^T      X = A [rows, k],  Y = B,            out = C [rows, n]    */
  GEMM_GROUPED_GRAD_A = 1,  /* dA[i] = dC[i] . B[e]      X = dC [rows, n], Y = B,            out = dA [rows, k]   */
  GEMM_GROUPED_GRAD_B = 2   /* dB[e] = sum dC[i]^T A[i]  X = dC [rows, n], Y = A [rows, k],  out = dB [E, n, k]   */
} gemm_grouped_mode_t;

/*
 * One grouped product, row i of expert e throughout: sizes, types and layout. B and dB are
 * [experts, n, k] with row stride ldy (GRAD_B: ldo) and `stride` elements between experts.
 */
typedef struct {
  gemm_grouped_mode_t mode;
  int64_t rows, experts, n, k;
  gemm_dtype_t in_dtype;  /* F16 or BF16, X and Y alike */
  gemm_dtype_t out_dtype; /* F16, BF16 or F32 */
  int64_t ldx, ldy, ldo, stride;
  int zero_rest; /* FORWARD, GRAD_A: zero the output rows that belong to no expert, else leave them */
  int tile;      /* rows of an output tile: 0 for the library's choice, else 32 (not GRAD_B), 128 or 256 */
} gemm_grouped_t;

/*
 * fp32 sums, rounded once. GRAD_B writes every expert's gradient, zeros for one without rows. The
 * sums run in a fixed order: results do not change from run to run.
 *   Any element alignment and row length will do. The 256-row tiles want whole 16-byte chunks: where they
 * are chosen, an operand whose base, row length, leading dimension or expert stride is not a multiple of
 * 16 bytes is first copied to padded rows in the workspace. 32-row tiles cut a long sum of few tiles into parts,
 * fp32 planes in the workspace that a second kernel adds in their order.
 * Errors: GEMM_ERR_INVALID (null pointer, bad enum, negative size, ld or stride too small, workspace
 *         too small), GEMM_ERR_UNSUPPORTED (types; rows beyond 2^31 - 1; experts beyond 2^24; more than
 *         2^24 output tiles; a leading dimension of 2^20 elements or more; experts times stride beyond
 *         2^54 elements), GEMM_ERR_HIP.
 */
gemm_status_t gemm_grouped_workspace_bytes(const gemm_grouped_t* p, const void* X, const void* Y, int64_t* out);
gemm_status_t gemm_grouped_run(const gemm_grouped_t* p, const void* X, const void* Y, void* out,
                               const int32_t* offsets, void* workspace, int64_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------ 4-bit weights */

/*
 * `matrices` weight matrices [n, k] of 4-bit values q with one scale (and, with has_zeros, one zero
 * point) per group of `group` (32, 64 or 128) neighbouring k; the last group may be short. The weight
 * is (q - z) * s, z = 8 without zero points.
 *
 * gemm_w4_pack lays them out for gemm_w4_run, once: q is [matrices, n, k] with one value per byte
 * (the low four bits), scales [matrices, n, ceil(k / group)] 16-bit, zeros the same shape in bytes
 * (low four bits) or NULL, all contiguous; `packed` is gemm_w4_packed_bytes long and 16-byte aligned.
 * Errors: GEMM_ERR_INVALID, GEMM_ERR_UNSUPPORTED (group; matrices, n or k beyond 2^24; more than 2^45
 *         blocks of 16 n by 128 k), GEMM_ERR_HIP.
 */
gemm_status_t gemm_w4_packed_bytes(int64_t matrices, int64_t n, int64_t k, int group, int has_zeros, int64_t* out);
gemm_status_t gemm_w4_pack(const uint8_t* q, const void* scales, const uint8_t* zeros, int64_t matrices, int64_t n,
                           int64_t k, int group, void* packed, void* stream);

/*
 * out[i] = x[i] . W[e]^T with row i's matrix: matrix 0 for all rows with offsets NULL (matrices = 1),
 * else expert e's (matrices = E). x [rows, k] and the scales are `dtype` (F16 or BF16); out_dtype F16,
 * BF16 or F32. q - z is exact in either type, so no weight is rounded: products are exact, each
 * group's sum is fp32 and multiplied by its scale in fp32 (the sum of x * (q - z) over a group has to
 * stay inside fp32's range), and the result is rounded once. Rows that belong to no expert: zero_rest
 * as above. With few columns the sum over k is split over workgroups, into planes in the workspace.
 * Errors: GEMM_ERR_INVALID, GEMM_ERR_UNSUPPORTED (types; group; a weight that gemm_w4_pack refuses; ldx of
 *         2^23 or more; more than 65535 blocks of 64 rows: 4194240 rows of one matrix, and with offsets
 *         (rows - g) / 64 + g blocks, g = min(matrices + 2, rows)), GEMM_ERR_HIP.
 */
typedef struct {
  int64_t rows, matrices, n, k;
  int group, has_zeros;
  gemm_dtype_t dtype, out_dtype;
  int64_t ldx, ldo;
  int zero_rest;
} gemm_w4_t;
gemm_status_t gemm_w4_workspace_bytes(const gemm_w4_t* p, int has_offsets, int64_t* out);
gemm_status_t gemm_w4_run(const gemm_w4_t* p, const void* x, const void* packed, const int32_t* offsets, void* out,
                          void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPT_EXPERTS_H */
