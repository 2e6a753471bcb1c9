// C ABI of the calls in include/moe_int4_block.h: like api.cpp, every
// argument is checked on the host, without a HIP call, before anything is
// enqueued.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "api_internal.h"
#include "launch.h"
#include "moe_int4_block.h"

namespace {

using moe::aligned;
using moe::hip_status;
using moe::kWorkspaceAlign;

constexpr int kMaxExperts = 1024;
constexpr int kMaxPositions = 1 << 24;
constexpr int kMaxCols = 65536;
constexpr int kMaxRowsDiv = 256;
constexpr int kMaxSwiglu = 32768;
constexpr int kMaxNorm = 8192;

bool float_dtype(moe_dtype t) { return t == MOE_F32 || t == MOE_BF16; }

// Sizes of a grouped product; `k_step`: K's multiple.
moe_status check_sizes(int32_t E, int32_t P, int32_t N, int32_t K, int k_step) {
  if (E <= 0 || P < 0 || N <= 0 || K <= 0 || N % 8 != 0 || K % k_step != 0) return MOE_ERR_SHAPE;
  if (E > kMaxExperts || P > kMaxPositions || N > kMaxCols || K > kMaxCols)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// The gathered operand's rows.
moe_status check_rows(int32_t P, int32_t x_rows, const int32_t* rows, int32_t rows_div) {
  if (x_rows < 0 || rows_div < 1) return MOE_ERR_SHAPE;
  if (!rows && P > 0 && (x_rows < P || rows_div != 1)) return MOE_ERR_SHAPE;
  if (rows_div > kMaxRowsDiv || static_cast<int64_t>(x_rows) * rows_div > kMaxPositions)
    return MOE_ERR_UNSUPPORTED;
  return aligned(rows, 4) ? MOE_OK : MOE_ERR_ALIGN;
}

void set_rows(moe::GroupedMm& g, int32_t x_rows, const int32_t* rows, int32_t rows_div) {
  g.rows = rows;
  g.row_limit = static_cast<uint32_t>(x_rows) * static_cast<uint32_t>(rows_div);
  g.div_magic = rows_div == 1 ? 0u
                              : static_cast<uint32_t>(((uint64_t(1) << 32) + rows_div - 1) /
                                                      static_cast<uint32_t>(rows_div));
}

moe_status check_norm(int32_t T, int32_t d, const void* y, moe_dtype y_dt, const float* w_post,
                      const void* gate, int32_t gate_rows, float scale, const void* res,
                      moe_dtype res_dt, const float* w_pre, float eps, moe_dtype normed_dt) {
  if (T < 0 || d <= 0 || d % 8 != 0) return MOE_ERR_SHAPE;
  if (d > kMaxNorm || T > kMaxPositions) return MOE_ERR_UNSUPPORTED;
  if (!float_dtype(y_dt) || !float_dtype(res_dt) || !float_dtype(normed_dt)) return MOE_ERR_DTYPE;
  if (!isfinite(scale) || !isfinite(eps) || !(eps > 0.0f)) return MOE_ERR_SHAPE;
  if (gate ? (gate_rows != 1 && gate_rows != T) : gate_rows != 0) return MOE_ERR_SHAPE;
  if (!aligned(y, 16) || !aligned(res, 16) || !aligned(gate, 16) || !aligned(w_post, 16) ||
      !aligned(w_pre, 16))
    return MOE_ERR_ALIGN;
  if (T > 0 && !y && (!res || w_post || gate)) return MOE_ERR_NULL;
  return MOE_OK;
}

moe::BlockNorm norm_args(int32_t T, int32_t d, const void* y, moe_dtype y_dt, const float* w_post,
                         const void* gate, int32_t gate_rows, float scale, const void* res,
                         moe_dtype res_dt, const float* w_pre, float eps, moe_dtype normed_dt) {
  moe::BlockNorm g{};
  g.T = T;
  g.d = d;
  g.gate_rows = gate_rows;
  g.scale = scale;
  g.eps = eps;
  g.y_bf16 = y_dt == MOE_BF16;
  g.res_bf16 = res_dt == MOE_BF16;
  g.normed_bf16 = normed_dt == MOE_BF16;
  g.y = y;
  g.res = res;
  g.gate = gate;
  g.w_post = w_post;
  g.w_pre = w_pre;
  return g;
}

}  // namespace

extern "C" {

moe_status moe_grouped_mm(int32_t E, int32_t P, int32_t N, int32_t K, const void* x,
                          int32_t x_rows, const int32_t* rows, int32_t rows_div, const void* w,
                          const int32_t* offsets, void* y, moe_dtype y_dt, void* stream) {
  moe_status st = check_sizes(E, P, N, K, 8);
  if (st != MOE_OK) return st;
  if (!float_dtype(y_dt)) return MOE_ERR_DTYPE;
  if ((st = check_rows(P, x_rows, rows, rows_div)) != MOE_OK) return st;
  if (P == 0) return MOE_OK;
  if ((!x && x_rows > 0) || !w || !offsets || !y) return MOE_ERR_NULL;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(y, 16) || !aligned(offsets, 4))
    return MOE_ERR_ALIGN;
  moe::GroupedMm g{};
  g.r = static_cast<const uint8_t*>(x);
  g.f = static_cast<const uint8_t*>(w);
  g.offsets = offsets;
  set_rows(g, x_rows, rows, rows_div);
  g.out = y;
  g.E = E;
  g.P = P;
  g.N = N;
  g.K = K;
  g.out_f32 = y_dt == MOE_F32;
  return hip_status(
      moe::launch_grouped_mm(g, moe::kGroupedRows, static_cast<hipStream_t>(stream)));
}

moe_status moe_grouped_mm_dx(int32_t E, int32_t P, int32_t N, int32_t K, const void* dy,
                             const void* w, const int32_t* offsets, void* dx, moe_dtype dx_dt,
                             void* stream) {
  const moe_status st = check_sizes(E, P, N, K, 8);
  if (st != MOE_OK) return st;
  if (!float_dtype(dx_dt)) return MOE_ERR_DTYPE;
  if (P == 0) return MOE_OK;
  if (!dy || !w || !offsets || !dx) return MOE_ERR_NULL;
  if (!aligned(dy, 16) || !aligned(w, 16) || !aligned(dx, 16) || !aligned(offsets, 4))
    return MOE_ERR_ALIGN;
  moe::GroupedMm g{};
  g.r = static_cast<const uint8_t*>(dy);
  g.f = static_cast<const uint8_t*>(w);
  g.offsets = offsets;
  g.out = dx;
  g.E = E;
  g.P = P;
  g.N = N;
  g.K = K;
  g.out_f32 = dx_dt == MOE_F32;
  return hip_status(
      moe::launch_grouped_mm(g, moe::kGroupedInput, static_cast<hipStream_t>(stream)));
}

size_t moe_grouped_mm_dw_workspace_bytes(int32_t E, int32_t P, int32_t N, int32_t K) {
  if (check_sizes(E, P, N, K, 8) != MOE_OK) return 0;
  return moe::round_up(moe::grouped_dw_workspace(E, P, N, K));
}

moe_status moe_grouped_mm_dw(int32_t E, int32_t P, int32_t N, int32_t K, const void* dy,
                             const void* x, int32_t x_rows, const int32_t* rows, int32_t rows_div,
                             const int32_t* offsets, void* dw, moe_dtype dw_dt, void* workspace,
                             size_t workspace_bytes, void* stream) {
  moe_status st = check_sizes(E, P, N, K, 8);
  if (st != MOE_OK) return st;
  if (!float_dtype(dw_dt)) return MOE_ERR_DTYPE;
  if ((st = check_rows(P, x_rows, rows, rows_div)) != MOE_OK) return st;
  const size_t need = moe_grouped_mm_dw_workspace_bytes(E, P, N, K);
  if (!offsets || !dw || (need > 0 && !workspace)) return MOE_ERR_NULL;
  if (P > 0 && (!dy || (!x && x_rows > 0))) return MOE_ERR_NULL;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(dw, 16) || !aligned(offsets, 4) ||
      !aligned(workspace, kWorkspaceAlign))
    return MOE_ERR_ALIGN;
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
  moe::GroupedMm g{};
  g.r = static_cast<const uint8_t*>(dy);
  g.f = static_cast<const uint8_t*>(x);
  g.offsets = offsets;
  set_rows(g, x_rows, rows, rows_div);
  g.out = dw;
  g.workspace = workspace;
  g.E = E;
  g.P = P;
  g.N = N;
  g.K = K;
  g.out_f32 = dw_dt == MOE_F32;
  return hip_status(
      moe::launch_grouped_mm(g, moe::kGroupedWeights, static_cast<hipStream_t>(stream)));
}

moe_status moe_blockscale_quantize(int32_t n_mats, int32_t R, int32_t K, const void* x,
                                   moe_dtype x_dt, int32_t block_rows, uint8_t* codes,
                                   float* scales, void* stream) {
  if (n_mats < 0 || R < 0 || K <= 0 || K % 16 != 0) return MOE_ERR_SHAPE;
  if (K > kMaxCols || (block_rows != 1 && block_rows != 128)) return MOE_ERR_UNSUPPORTED;
  const int64_t rows = static_cast<int64_t>(n_mats) * R, kb = (K + 127) / 128;
  const int64_t blocks =
      block_rows == 1 ? rows * kb : n_mats * ((static_cast<int64_t>(R) + 127) / 128) * kb;
  if (rows > INT32_MAX || blocks > (block_rows == 1 ? int64_t(1) << 34 : int64_t(INT32_MAX)))
    return MOE_ERR_UNSUPPORTED;
  if (!float_dtype(x_dt)) return MOE_ERR_DTYPE;
  if (rows == 0) return MOE_OK;
  if (!x || !codes || !scales) return MOE_ERR_NULL;
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return MOE_ERR_ALIGN;
  return hip_status(moe::launch_blockscale_quantize(n_mats, R, K, x, x_dt == MOE_F32,
                                                    block_rows == 128, codes, scales,
                                                    static_cast<hipStream_t>(stream)));
}

moe_status moe_blockscale_mm(int32_t E, int32_t P, int32_t N, int32_t K, const uint8_t* xq,
                             const float* xs, int32_t x_rows, const int32_t* rows,
                             int32_t rows_div, const uint8_t* wq, const float* ws,
                             const int32_t* offsets, void* y, moe_dtype y_dt, void* stream) {
  moe_status st = check_sizes(E, P, N, K, 16);
  if (st != MOE_OK) return st;
  if (!float_dtype(y_dt)) return MOE_ERR_DTYPE;
  if ((st = check_rows(P, x_rows, rows, rows_div)) != MOE_OK) return st;
  if (P == 0) return MOE_OK;
  if (((!xq || !xs) && x_rows > 0) || !wq || !ws || !offsets || !y) return MOE_ERR_NULL;
  if (!aligned(xq, 16) || !aligned(wq, 16) || !aligned(y, 16) || !aligned(xs, 4) ||
      !aligned(ws, 4) || !aligned(offsets, 4))
    return MOE_ERR_ALIGN;
  moe::GroupedMm g{};
  g.r = xq;
  g.f = wq;
  g.r_scale = xs;
  g.f_scale = ws;
  g.offsets = offsets;
  set_rows(g, x_rows, rows, rows_div);
  g.out = y;
  g.E = E;
  g.P = P;
  g.N = N;
  g.K = K;
  g.out_f32 = y_dt == MOE_F32;
  return hip_status(
      moe::launch_grouped_mm(g, moe::kGroupedCodes, static_cast<hipStream_t>(stream)));
}

namespace {
moe_status check_swiglu(int32_t P, int32_t f, moe_dtype dt, const int32_t* n_rows, int f_step) {
  if (P < 0 || f <= 0 || f % f_step != 0) return MOE_ERR_SHAPE;
  if (P > kMaxPositions || f > kMaxSwiglu) return MOE_ERR_UNSUPPORTED;
  if (!float_dtype(dt)) return MOE_ERR_DTYPE;
  return aligned(n_rows, 4) ? MOE_OK : MOE_ERR_ALIGN;
}
}  // namespace

moe_status moe_swiglu(int32_t P, int32_t f, const void* gu, void* h, moe_dtype dt,
                      const int32_t* n_rows, void* stream) {
  const moe_status st = check_swiglu(P, f, dt, n_rows, 8);
  if (st != MOE_OK || P == 0) return st;
  if (!gu || !h) return MOE_ERR_NULL;
  if (!aligned(gu, 16) || !aligned(h, 16)) return MOE_ERR_ALIGN;
  return hip_status(moe::launch_swiglu(P, f, gu, dt == MOE_F32, h, nullptr, n_rows,
                                       static_cast<hipStream_t>(stream)));
}

moe_status moe_swiglu_quantize(int32_t P, int32_t f, const void* gu, moe_dtype dt, uint8_t* codes,
                               float* scales, const int32_t* n_rows, void* stream) {
  const moe_status st = check_swiglu(P, f, dt, n_rows, 16);
  if (st != MOE_OK || P == 0) return st;
  if (!gu || !codes || !scales) return MOE_ERR_NULL;
  if (!aligned(gu, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return MOE_ERR_ALIGN;
  return hip_status(moe::launch_swiglu(P, f, gu, dt == MOE_F32, codes, scales, n_rows,
                                       static_cast<hipStream_t>(stream)));
}

moe_status moe_swiglu_grad(int32_t P, int32_t f, const void* gu, const void* dh, void* dgu,
                           moe_dtype dt, const int32_t* n_rows, void* stream) {
  const moe_status st = check_swiglu(P, f, dt, n_rows, 8);
  if (st != MOE_OK || P == 0) return st;
  if (!gu || !dh || !dgu) return MOE_ERR_NULL;
  if (!aligned(gu, 16) || !aligned(dh, 16) || !aligned(dgu, 16)) return MOE_ERR_ALIGN;
  return hip_status(moe::launch_swiglu_grad(P, f, gu, dh, dt == MOE_F32, dgu, n_rows,
                                            static_cast<hipStream_t>(stream)));
}

moe_status moe_combine_grad(const moe_shape* shape, int32_t T, const void* dout, moe_dtype out_dt,
                            const void* y, moe_dtype y_dt, const int32_t* inv_perm,
                            const float* topk_w, void* dy, float* dtopk_w, void* stream) {
  const moe_status st = moe::combine_check(shape, T, y_dt, out_dt);
  if (st != MOE_OK || T == 0) return st;
  if (!dout || !y || !inv_perm || !topk_w || !dy || !dtopk_w) return MOE_ERR_NULL;
  if (!aligned(dout, 16) || !aligned(y, 16) || !aligned(dy, 16) || !aligned(inv_perm, 4) ||
      !aligned(topk_w, 4) || !aligned(dtopk_w, 4))
    return MOE_ERR_ALIGN;
  return hip_status(moe::launch_combine_grad(T, shape->d, shape->top_k, dout, out_dt == MOE_BF16,
                                             y, y_dt == MOE_BF16, inv_perm, topk_w, dy, dtopk_w,
                                             static_cast<hipStream_t>(stream)));
}

moe_status moe_block_norm(int32_t T, int32_t d, const void* y, moe_dtype y_dt,
                          const float* w_post, const void* gate, int32_t gate_rows, float scale,
                          const void* res, moe_dtype res_dt, void* res_out, const float* w_pre,
                          float eps, void* normed, moe_dtype normed_dt, void* stream) {
  const moe_status st = check_norm(T, d, y, y_dt, w_post, gate, gate_rows, scale, res, res_dt,
                                   w_pre, eps, normed_dt);
  if (st != MOE_OK || T == 0) return st;
  if ((w_pre != nullptr) != (normed != nullptr) || (!res_out && !normed)) return MOE_ERR_NULL;
  if (!aligned(res_out, 16) || !aligned(normed, 16)) return MOE_ERR_ALIGN;
  moe::BlockNorm g = norm_args(T, d, y, y_dt, w_post, gate, gate_rows, scale, res, res_dt, w_pre,
                               eps, normed_dt);
  g.res_out = res_out;
  g.normed = normed;
  return hip_status(moe::launch_block_norm(g, static_cast<hipStream_t>(stream)));
}

size_t moe_block_norm_grad_workspace_bytes(int32_t T, int32_t d) {
  if (T < 0 || d <= 0 || d % 8 != 0 || d > kMaxNorm || T > kMaxPositions) return 0;
  return moe::round_up(static_cast<size_t>(moe::norm_grad_parts(T, d)) * 2 * d * sizeof(float));
}

moe_status moe_block_norm_grad(int32_t T, int32_t d, const void* y, moe_dtype y_dt,
                               const float* w_post, const void* gate, int32_t gate_rows,
                               float scale, const void* res, moe_dtype res_dt, const float* w_pre,
                               float eps, const void* dr, const void* dn, moe_dtype normed_dt,
                               void* dy, void* dres, void* dgate, float* dw_post, float* dw_pre,
                               void* workspace, size_t workspace_bytes, void* stream) {
  const moe_status st = check_norm(T, d, y, y_dt, w_post, gate, gate_rows, scale, res, res_dt,
                                   w_pre, eps, normed_dt);
  if (st != MOE_OK) return st;
  if (T > 0 && (w_pre != nullptr) != (dn != nullptr)) return MOE_ERR_NULL;
  if ((!w_post && dw_post) || (!w_pre && dw_pre) || (!gate && dgate) || (T > 0 && !y && dy))
    return MOE_ERR_NULL;
  if (!aligned(dr, 16) || !aligned(dn, 16) || !aligned(dy, 16) || !aligned(dres, 16) ||
      !aligned(dgate, 16) || !aligned(dw_post, 4) || !aligned(dw_pre, 4) ||
      !aligned(workspace, kWorkspaceAlign))
    return MOE_ERR_ALIGN;
  const bool columns = dw_post || dw_pre || (dgate && gate_rows == 1);
  const size_t need = columns ? moe_block_norm_grad_workspace_bytes(T, d) : 0;
  if (need > 0 && !workspace) return MOE_ERR_NULL;
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
  if (!columns && (T == 0 || (!dy && !dres && !dgate))) return MOE_OK;
  moe::BlockNorm g = norm_args(T, d, y, y_dt, w_post, gate, gate_rows, scale, res, res_dt, w_pre,
                               eps, normed_dt);
  g.dr = dr;
  g.dn = dn;
  g.dy = dy;
  g.dres = dres;
  g.dgate = dgate;
  g.dw_post = dw_post;
  g.dw_pre = dw_pre;
  g.part = columns ? static_cast<float*>(workspace) : nullptr;
  g.columns = columns;
  return hip_status(moe::launch_block_norm_grad(g, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
