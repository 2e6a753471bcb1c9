/*
 * moe_int4_block.h -- the layer on float and 8-bit expert weights, its
 * gradients, and the norms around it.
 *
 * moe_int4.h serves the layer from int4 / MXFP4 expert blocks.  The calls here
 * compute the same layer from the weights a checkpoint has before that
 * conversion (bfloat16, or e4m3 codes with a float32 scale per 128 x 128) or as
 * 8-bit integers (with a float32 scale per output channel), and train it:
 *
 *   moe_grouped_mm        y[p] = W_e x[row(p)] over rows grouped by expert
 *   moe_grouped_mm_dx     its input's gradient
 *   moe_grouped_mm_dw     its weights' gradient
 *   moe_blockscale_quantize  bf16 / f32 -> e4m3 codes and block scales
 *   moe_blockscale_mm     moe_grouped_mm over e4m3 codes
 *   moe_rowscale_quantize bf16 / f32 -> 8-bit integers and a scale per row
 *   moe_rowscale_mm       moe_grouped_mm over 8-bit integers
 *   moe_swiglu[_quantize, _rowscale] silu(gate) * up between the two products
 *   moe_swiglu_grad       its gradient
 *   moe_combine_grad      moe_combine's gradient
 *   moe_block_norm        post norm, gate, residual and next pre norm in one pass
 *   moe_block_norm_grad   its gradient
 *
 * Conventions as in moe_int4.h: device pointers owned by the caller, work
 * enqueued on `stream`, nothing allocated, no state, arguments checked before
 * anything is enqueued.  Results do not depend on the order in which
 * workgroups run (no atomics), so a call repeated on the same inputs gives the
 * same bits (a product's last bits may differ between calls of other sizes, which
 * other kernels add up in another order).  Tensors are row-major without gaps;
 * bf16 and f32 arrays are 16-byte aligned, codes, the norms' weights and the
 * scales of a matrix's output channels too, int32 arrays, other scales and the
 * weights' gradients of the norms 4-byte.
 *
 * Rows grouped by expert: position p belongs to expert e when
 *   offsets[e] <= p < offsets[e + 1],
 * offsets [E + 1] as moe_union writes it (moe_union's perm is `rows` with
 * rows_div = top_k).  P is the number of positions the arrays hold; positions
 * at or past offsets[E] belong to no expert and their output rows are left as
 * they were.  offsets are read on the device and clamped to [0, P] there.
 * E = 1 with offsets {0, P} is a plain product (the shared expert).
 * Limits: 1 <= E <= 1024, 0 <= P <= 2^24 (else MOE_ERR_SHAPE where negative or
 * zero, MOE_ERR_UNSUPPORTED where larger); P == 0 enqueues nothing, except
 * that moe_grouped_mm_dw writes its zeros.
 */
#ifndef MOE_INT4_BLOCK_H
#define MOE_INT4_BLOCK_H

#include "moe_int4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows times an expert's weights:
 *   y[p][n] = sum_k w[e][n][k] * x[row(p)][k],   row(p) = rows ? rows[p] / rows_div : p
 * summed in float32 on the bf16 matrix cores, rounded once to y's type.
 *  N, K      output and input columns; multiples of 8, 8..65536
 *  x         [x_rows][K] bf16; x_rows >= P without rows
 *  rows      [P] int32 or NULL; an entry outside [0, x_rows * rows_div) stands
 *            for a row of zeros (its results are zeros, NaN where the weights
 *            are not finite).  x_rows * rows_div <= 2^24
 *  rows_div  1..256 (1 without rows, unless P is 0)
 *  w         [E][N][K] bf16
 *  y         out [P][N], bf16 or f32; must not overlap an input */
moe_status moe_grouped_mm(int32_t E, int32_t P, int32_t N, int32_t K, const void* x,
                          int32_t x_rows, const int32_t* rows, int32_t rows_div, const void* w,
                          const int32_t* offsets, void* y, moe_dtype y_dt, void* stream);

/* Gradient of moe_grouped_mm's input, by position (before any gather):
 *   dx[p][k] = sum_n dy[p][n] * w[e][n][k]
 * The gradient of a gathered x sums a row's positions: moe_combine with weights
 * of 1 does that.
 *  dy [P][N] bf16, w [E][N][K] bf16, dx out [P][K] bf16 or f32. */
moe_status moe_grouped_mm_dx(int32_t E, int32_t P, int32_t N, int32_t K, const void* dy,
                             const void* w, const int32_t* offsets, void* dx, moe_dtype dx_dt,
                             void* stream);

/* Scratch bytes of moe_grouped_mm_dw; 0 for sizes the call rejects. */
size_t moe_grouped_mm_dw_workspace_bytes(int32_t E, int32_t P, int32_t N, int32_t K);

/* Gradient of moe_grouped_mm's weights:
 *   dw[e][n][k] = sum over e's positions p of dy[p][n] * x[row(p)][k]
 * Every expert's dw is written; one without positions gets zeros.
 *  dy [P][N] bf16; x, x_rows, rows, rows_div as in moe_grouped_mm;
 *  dw out [E][N][K] bf16 or f32
 *  workspace >= moe_grouped_mm_dw_workspace_bytes(E, P, N, K), 256-byte aligned,
 *            no initial contents required; never shared between calls that may
 *            run at the same time */
moe_status moe_grouped_mm_dw(int32_t E, int32_t P, int32_t N, int32_t K, const void* dy,
                             const void* x, int32_t x_rows, const int32_t* rows, int32_t rows_div,
                             const int32_t* offsets, void* dw, moe_dtype dw_dt, void* workspace,
                             size_t workspace_bytes, void* stream);

/* e4m3 codes (OCP FP8: 4 exponent bits, bias 7, largest 448) with a float32
 * scale per block: value = code * scale.
 *   scale = 2^n, the smallest n >= -126 with absmax <= 448 * 2^n over the
 *           block's finite values (1 for a block of zeros)
 *   code  = the e4m3 value nearest to x / scale, ties to even (the division is
 *           exact, so the code is decided exactly); NaN for a non-finite x
 *  n_mats, R, K  matrices [R][K] back to back; K a multiple of 16, 16..65536
 *  block_rows    1: a block is 128 columns of a row, scales [n_mats][R][ceil(K/128)];
 *                128: 128 rows by 128 columns of one matrix,
 *                scales [n_mats][ceil(R/128)][ceil(K/128)].  Blocks at an edge are
 *                short.  Anything else is MOE_ERR_UNSUPPORTED.
 * n_mats * R <= 2^31 - 1; at most 2^31 - 1 blocks of 128 x 128 and 2^34 of 1 x 128. */
moe_status moe_blockscale_quantize(int32_t n_mats, int32_t R, int32_t K, const void* x,
                                   moe_dtype x_dt, int32_t block_rows, uint8_t* codes,
                                   float* scales, void* stream);

/* moe_grouped_mm over e4m3 codes:
 *   y[p][n] = sum_b xs[row(p)][b] * ws[e][n / 128][b] *
 *             sum over k in block b of wq[e][n][k] * xq[row(p)][k]
 * with any float32 scales (not only moe_blockscale_quantize's); the product of
 * the two scales is taken first, in float32, so it is to be finite.
 *  N a multiple of 8 and K of 16, 16..65536
 *  xq [x_rows][K], xs [x_rows][ceil(K/128)], wq [E][N][K],
 *  ws [E][ceil(N/128)][ceil(K/128)]; rows as in moe_grouped_mm
 *  y  out [P][N].  The codes are multiplied as bf16, which holds every e4m3
 *     value: products are exact, and summed in float32 for either type of y. */
moe_status moe_blockscale_mm(int32_t E, int32_t P, int32_t N, int32_t K, const uint8_t* xq,
                             const float* xs, int32_t x_rows, const int32_t* rows,
                             int32_t rows_div, const uint8_t* wq, const float* ws,
                             const int32_t* offsets, void* y, moe_dtype y_dt, void* stream);

/* 8-bit integers with a float32 scale per row (a token, or an output channel of a
 * weight matrix): value = code * scale.
 *   scale = max(absmax * c, 2^-126), c = 1 / 127 and the product rounded to float32;
 *           1 for a row of zeros, NaN for one that holds a value that is not finite
 *   code  = the integer nearest to x / scale, ties to even, -127..127, decided
 *           exactly; 0 where the scale is NaN
 *  rows    0..2^31 - 1 (n matrices of R rows: n * R); K a multiple of 16, 16..65536
 *  x       [rows][K] bf16 or f32; codes [rows][K], scales [rows] */
moe_status moe_rowscale_quantize(int32_t rows, int32_t K, const void* x, moe_dtype x_dt,
                                 int8_t* codes, float* scales, void* stream);

/* moe_grouped_mm over 8-bit integers:
 *   y[p][n] = (sum_k wq[e][n][k] * xq[row(p)][k]) * xs[row(p)] * ws[e][n]
 * with any codes and float32 scales; the sum is exact (int32), then rounded to
 * float32, as is each product with a scale, and the result to y's type.
 *  N a multiple of 8 and K of 16, 16..65536
 *  xq [x_rows][K], xs [x_rows], wq [E][N][K], ws [E][N] (16-byte aligned); rows as in
 *  moe_grouped_mm, a row of zeros having a scale of 0;  y out [P][N] */
moe_status moe_rowscale_mm(int32_t E, int32_t P, int32_t N, int32_t K, const int8_t* xq,
                           const float* xs, int32_t x_rows, const int32_t* rows, int32_t rows_div,
                           const int8_t* wq, const float* ws, const int32_t* offsets, void* y,
                           moe_dtype y_dt, void* stream);

/* h[p][c] = silu(gu[p][c]) * gu[p][f + c] for p < P, silu(z) = z / (1 + e^-z).
 *  f       a multiple of 8, 8..32768
 *  gu, h   [P][2 f] and [P][f], both dt (bf16 or f32)
 *  n_rows  device int32, or NULL: rows from *n_rows on are left as they were
 *          (moe_union's offsets + E) */
moe_status moe_swiglu(int32_t P, int32_t f, const void* gu, void* h, moe_dtype dt,
                      const int32_t* n_rows, void* stream);

/* moe_swiglu, then moe_blockscale_quantize's 1 x 128 blocks of the float32
 * result: codes [P][f], scales [P][ceil(f/128)]; f a multiple of 16. */
moe_status moe_swiglu_quantize(int32_t P, int32_t f, const void* gu, moe_dtype dt, uint8_t* codes,
                               float* scales, const int32_t* n_rows, void* stream);

/* moe_swiglu, then moe_rowscale_quantize of the float32 result: codes [P][f],
 * scales [P]; f a multiple of 16. */
moe_status moe_swiglu_rowscale(int32_t P, int32_t f, const void* gu, moe_dtype dt, int8_t* codes,
                               float* scales, const int32_t* n_rows, void* stream);

/* With s = 1 / (1 + e^-g): dgu[p][c] = dh u s (1 + g (1 - s)) and
 * dgu[p][f + c] = dh g s.  dgu [P][2 f] may be gu itself. */
moe_status moe_swiglu_grad(int32_t P, int32_t f, const void* gu, const void* dh, void* dgu,
                           moe_dtype dt, const int32_t* n_rows, void* stream);

/* Gradient of moe_combine, given dout [T][d] (out_dt) of its out:
 *   dy[inv_perm[s]]  = topk_w[s] * dout[t]         s = t * top_k + j
 *   dtopk_w[s]       = sum_c y[inv_perm[s]][c] * dout[t][c]
 * (the shared expert's rows have dout itself).  A slot with inv_perm outside
 * [0, T * top_k) has dtopk_w 0 and writes no row of dy.
 *  y   [T*top_k][d] (y_dt), grouped order; dy out, same type, may be y itself
 *  inv_perm as moe_union writes it: no position twice
 *  dtopk_w out [T][top_k] float32 */
moe_status moe_combine_grad(const moe_shape* shape, int32_t T, const void* dout, moe_dtype out_dt,
                            const void* y, moe_dtype y_dt, const int32_t* inv_perm,
                            const float* topk_w, void* dy, float* dtopk_w, void* stream);

/* What stands between one block's output y and the next block's input, in one
 * pass over each of T rows of d columns:
 *   p = y * w_post / sqrt(mean(y^2) + eps)        (p = y where w_post is NULL)
 *   r = res + scale * gate * p
 *   n = r * w_pre / sqrt(mean(r^2) + eps)         (none where w_pre is NULL)
 * The squares are summed in float32 (a row whose sum passes 3.4e38 is outside
 * the call's range); n is taken from r before r is rounded to res_dt.
 *  d       a multiple of 8, 8..8192
 *  y       [T][d] y_dt, or NULL (r = res; w_post and gate must be NULL too)
 *  gate    [gate_rows][d] y_dt, gate_rows 1 (one vector for all rows) or T; NULL
 *          for none (gate_rows 0)
 *  res     [T][d] res_dt, or NULL for zeros (not where y is NULL)
 *  res_out out [T][d] res_dt, may be res itself; NULL if not wanted
 *  w_post, w_pre  [d] float32
 *  normed  out [T][d] normed_dt, exactly where w_pre is given
 *  eps     finite, > 0; scale finite (else MOE_ERR_SHAPE)
 * At least one of res_out and normed. */
moe_status moe_block_norm(int32_t T, int32_t d, const void* y, moe_dtype y_dt,
                          const float* w_post, const void* gate, int32_t gate_rows, float scale,
                          const void* res, moe_dtype res_dt, void* res_out, const float* w_pre,
                          float eps, void* normed, moe_dtype normed_dt, void* stream);

/* Scratch bytes of moe_block_norm_grad; 0 for sizes the call rejects. */
size_t moe_block_norm_grad_workspace_bytes(int32_t T, int32_t d);

/* Gradient of moe_block_norm at the same inputs, given dr [T][d] (res_dt, of
 * res_out; NULL for zeros) and dn [T][d] (normed_dt, of normed; exactly where
 * w_pre is given):
 *  dy      out [T][d] y_dt             dres  out [T][d] res_dt
 *  dgate   out [gate_rows][d] y_dt (summed over the rows of a gate of one row)
 *  dw_post, dw_pre  out [d] float32
 * Each output may be NULL, and must be where its input is (dres without res is
 * allowed: it is the gradient of r).  dy may be y and dres may be dr or res
 * itself; no other overlap.
 *  workspace >= moe_block_norm_grad_workspace_bytes(T, d), 256-byte aligned; never
 *            shared between calls that may run at the same time.  Needed only
 *            where dw_post, dw_pre or the dgate of a one-row gate is asked for
 *            (else it may be NULL).
 * T == 0 writes zeros to dw_post, dw_pre and a one-row dgate. */
moe_status moe_block_norm_grad(int32_t T, int32_t d, const void* y, moe_dtype y_dt,
                               const float* w_post, const void* gate, int32_t gate_rows,
                               float scale, const void* res, moe_dtype res_dt, const float* w_pre,
                               float eps, const void* dr, const void* dn, moe_dtype normed_dt,
                               void* dy, void* dres, void* dgate, float* dw_post, float* dw_pre,
                               void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_INT4_BLOCK_H */
