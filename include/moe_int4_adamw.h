/*
 * moe_int4_adamw.h -- one AdamW step over many tensors.
 *
 * The gradients that moe_int4_block.h computes, applied: all tensors of a layer
 * (or a model) in one call, with float32 or 8-bit moments.  Conventions as in
 * moe_int4.h: caller-owned device memory, work enqueued on `stream`, nothing
 * allocated, no state but the caller's, arguments checked before anything is
 * enqueued.  A step repeated on the same state with the same number gives the same
 * bits, however the tensors are listed.
 */
#ifndef MOE_INT4_ADAMW_H
#define MOE_INT4_ADAMW_H

#include "moe_int4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One tensor of n elements without gaps (n == 0: nothing is done for it).
 *  p         the parameter, f32 or bf16 (p_dt)
 *  master    float32 copy of a bf16 p, or NULL: the step then updates it and
 *            writes it, rounded to nearest even, to p (which is not read).
 *            Without one a bf16 p is itself updated in float32 and rounded, so a
 *            step smaller than half of p's last place is lost.
 *  g         its gradient, f32 or bf16 (g_dt), not written
 *  m, v      the moments: float32 [n] where the scales are NULL, else 8-bit codes
 *            [n] with a float32 scale per 256 consecutive elements, [ceil(n / 256)]
 * Every address is aligned for its element; where all of a tensor's are aligned
 * for four (16 bytes of float32, 8 of bf16, 4 of codes) the accesses are wide.
 * No array overlaps another one that the call writes.
 *
 * 8-bit moments.  m = e4m3 code * m_scale.  v = (root(c) * v_scale)^2, root(c) =
 * t * 2^e with e = max(c / 32 - 1, 0) and t = c - 32 e (0..63 in steps of 1, then 6
 * significant bits, up to 4032).  Scales are the smallest powers of two, 2^-126 at
 * least, that keep a block's largest |m| within 448 and largest sqrt(v) within 4032
 * (1 for a block of zeros); no code is 0 for a v that is not 0.  Codes and scales of
 * zero are moments of zero.
 *  Drawn codes, for beta2 = 0.999 among others: a code is one of the two next to
 *    its value, drawn by a hash of the step's number and the element's index in its
 *    tensor, so that the expected m and v are the values themselves.  Over 3000
 *    steps of normal, constant and 20 times shrinking gradients with beta2 from
 *    0.95 to 0.9999 the updates' norm stays within 6% of the one with float32
 *    moments.  A single root strays by 6 to 8% of itself down to a thirtieth of its
 *    block's largest, by 32% at a thousandth; one below 1 / 4032 of it is held as
 *    that much or more.
 *  Nearest codes, ties to even, where beta2 <= 0.95 and 1 - beta2 is between a fifth
 *    and a half of 1 - beta1 (0.9 and 0.95 among them).  A moment that a step would
 *    move by less than half a place (m 3 to 6%, sqrt(v) 0.8 to 1.6%) stays where it is, so
 *    that updates come out 1% too large for normal gradients, and for ones that
 *    hardly change up to 12% too small (0.9 and 0.95) or too large; any beta2 just
 *    above 0.95 has drawn codes.
 * Where m is not finite its code is NaN.  Where v is not (g^2 past float32's largest
 * is enough), its code is 255 and its block's v_scale a NaN whose last 8 bits are the
 * biased exponent of the scale that the block's other codes, up to 254, have: such
 * an element's parameter is what it is with float32 moments, and no other element
 * changes (its m is held within 448 m_scale and does not count for that).  A v_scale
 * of any NaN whose last 8 bits are 0 makes the whole block NaN. */
typedef struct {
  int64_t n;
  void* p;
  float* master;
  const void* g;
  void* m;
  void* v;
  float* m_scales;
  float* v_scales;
  moe_dtype p_dt;
  moe_dtype g_dt;
} moe_adamw_tensor;

/* For every element, in float32 (each operation rounded; the powers in double):
 *   g' = grad_scale * g
 *   m  = beta1 m + (1 - beta1) g'       v = beta2 v + (1 - beta2) g'^2
 *   p  = p (1 - lr * weight_decay)
 *        - lr / (1 - beta1^t) * (m / (sqrt(v) / sqrt(1 - beta2^t) + eps))
 * The update takes m and v before they are rounded to codes.
 *  tensors     host array of n_tensors (0..2^20), read during the call; at most
 *              2^40 elements each
 *  step        device int64, the step's number t, 1 for the first (smaller ones
 *              count as 1); the caller advances it, in a captured graph too
 *  grad_scale  device float32, or NULL for 1 (a clipping factor, or 1 / loss scale)
 *  lr, weight_decay  finite, >= 0; eps finite, > 0 in float32; beta1, beta2 in
 *              [0, 1) (else MOE_ERR_SHAPE); a captured step repeats these values and
 *              the tensors' addresses */
moe_status moe_adamw(const moe_adamw_tensor* tensors, int32_t n_tensors, const int64_t* step,
                     double lr, double beta1, double beta2, double eps, double weight_decay,
                     const float* grad_scale, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_INT4_ADAMW_H */
