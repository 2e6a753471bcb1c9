/*
 * moe_int4_few.h -- the whole layer for a few tokens on float and 8-bit experts.
 *
 * moe_layer_few computes what the calls of moe_int4_block.h compute in turn
 * (route, gate and up products, SwiGLU, down product, combine, shared expert)
 * for at most 32 tokens, in two kernels behind the router's (and a third that
 * joins partial sums where out is narrow), which read each hit expert's weights
 * once per 8 of its (token, expert) pairs for T <= 8, per 16 beyond.  Conventions as in
 * moe_int4_block.h: caller-owned device memory, work enqueued on `stream`, nothing
 * allocated, no state, arguments checked before anything is enqueued, no atomics in
 * memory: a call repeated on the same inputs gives the same bits.
 *
 * Against those calls it is the faster one up to 8 tokens (by 1.0 to 3 times), and with
 * more of them while an expert has fewer than about three: on e4m3 weights the
 * grouped products are up to 9% faster from there (32 tokens over 64 experts of
 * 2560 x 1024), on integers up to 3%, on bf16 from 24 tokens where d is 8192 (12%).
 */
#ifndef MOE_INT4_FEW_H
#define MOE_INT4_FEW_H

#include "moe_int4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How an expert's weights are held (always row-major without gaps):
 *  BF16  bfloat16
 *  E4M3  e4m3 codes with a float32 scale per 128 x 128, as moe_blockscale_mm's
 *  INT8  8-bit integers with a float32 scale per output channel, as
 *        moe_rowscale_mm's */
typedef enum {
  MOE_WEIGHTS_BF16 = 0,
  MOE_WEIGHTS_E4M3 = 1,
  MOE_WEIGHTS_INT8 = 2,
  MOE_WEIGHTS_INT_MIN_ = -2147483647 - 1,
  MOE_WEIGHTS_INT_MAX_ = 2147483647
} moe_weights;

/* The weights of n experts (the routed ones, or the shared one alone):
 *  gate_up         [n][2 f][d], an expert's gate rows first
 *  down            [n][d][f]
 *  gate_up_scales  E4M3 [n][ceil(2 f / 128)][ceil(d / 128)], INT8 [n][2 f], BF16 NULL
 *  down_scales     E4M3 [n][ceil(d / 128)][ceil(f / 128)], INT8 [n][d], BF16 NULL
 * weights 16-byte aligned, scales too for INT8 and 4-byte for E4M3. */
typedef struct {
  const void* gate_up;
  const void* down;
  const float* gate_up_scales;
  const float* down_scales;
} moe_expert_weights;

/* Scratch bytes of moe_layer_few; 0 for sizes the call rejects, and for T == 0. */
size_t moe_layer_few_workspace_bytes(const moe_shape* shape, int32_t T);

/* The layer for x [T][d] bf16:
 *   out[t] = sum_j topk_w[t][j] * FFN_e(x[t]), e = topk_idx[t][j], in the order of j
 *            (+ FFN_shared(x[t])),
 *   FFN_e(x) = D_e (silu(G_e x) * (U_e x)).
 *  shape     its group is not looked at beyond the values that moe_int4.h takes
 *  T         0..32 with T * top_k <= 256, else MOE_ERR_UNSUPPORTED; 0 enqueues nothing
 *  w_router  [E][d] float32: the routing is moe_route's (bias [E] or NULL) and is
 *            written to topk_idx and topk_w [T][top_k].  NULL: both are inputs (and
 *            bias is NULL); an id outside [0, E) contributes nothing, the same one
 *            twice counts twice, and an infinite weight gives an infinity or NaN.
 *  experts, shared  host structures of device addresses, read during the call;
 *            shared NULL exactly where the shape has no shared expert
 *  out       [T][d] bf16 or f32; must not overlap an input
 *  workspace >= moe_layer_few_workspace_bytes(shape, T), 256-byte aligned, no
 *            initial contents required; never shared between calls that may run
 *            at the same time
 * x is not rounded (unlike the calls on codes, which quantise it); the products
 * are summed in float32, and h = silu(G x) * (U x) is held between the kernels as a
 * sum of bf16 values: three for an out of f32 (all 24 bits), two for one of bf16
 * (17 bits, each off by 2^-17 of itself at most, where both are normal numbers).  A
 * bf16 out is thus off by 2^-17 sum |w D h| beside its own rounding, which is more
 * than half of its last place where that sum cancels by more than 2^8: an f32 out
 * does not have it.  Products with codes (up to 448 each) are summed before their
 * scales are multiplied in: a sum that passes float32's largest is an infinity,
 * also where the scaled result would not be. */
moe_status moe_layer_few(const moe_shape* shape, int32_t T, const void* x, const float* w_router,
                         const float* bias, moe_weights kind, const moe_expert_weights* experts,
                         const moe_expert_weights* shared, int32_t* topk_idx, float* topk_w,
                         void* out, moe_dtype out_dt, void* workspace, size_t workspace_bytes,
                         void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_INT4_FEW_H */
