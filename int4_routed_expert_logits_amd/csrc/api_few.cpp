// C ABI of include/moe_int4_few.h: like api.cpp, every argument is checked on
// the host, without a HIP call, before anything is enqueued.
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "api_internal.h"
#include "launch.h"
#include "moe_int4_few.h"

namespace {

using moe::aligned;
using moe::hip_status;
using moe::kWorkspaceAlign;

moe_status check_sizes(const moe_shape* shape, int32_t T) {
  const moe_status st = moe::combine_check(shape, T, MOE_F32, MOE_F32);
  if (st != MOE_OK) return st;
  if (T > moe::kFewTokens || T * shape->top_k > moe::kFewPairs) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_weights(const moe_expert_weights& w, moe_weights kind) {
  const bool codes = kind != MOE_WEIGHTS_BF16;
  if (!w.gate_up || !w.down || codes != (w.gate_up_scales != nullptr) ||
      codes != (w.down_scales != nullptr))
    return MOE_ERR_NULL;
  const size_t a = kind == MOE_WEIGHTS_INT8 ? 16 : 4;
  if (!aligned(w.gate_up, 16) || !aligned(w.down, 16) || !aligned(w.gate_up_scales, a) ||
      !aligned(w.down_scales, a))
    return MOE_ERR_ALIGN;
  return MOE_OK;
}

moe::FewScratch scratch_of(const moe_shape* s, int32_t T) {
  return moe::few_scratch(T, s->top_k, s->d, s->f, s->n_experts, s->f_shared != 0);
}

}  // namespace

extern "C" {

size_t moe_layer_few_workspace_bytes(const moe_shape* shape, int32_t T) {
  if (check_sizes(shape, T) != MOE_OK || T == 0) return 0;
  return moe_route_workspace_bytes(shape, T) +
         moe::round_up(scratch_of(shape, T).bytes);
}

moe_status moe_layer_few(const moe_shape* shape, int32_t T, const void* x, const float* w_router,
                         const float* bias, moe_weights kind, const moe_expert_weights* experts,
                         const moe_expert_weights* shared, int32_t* topk_idx, float* topk_w,
                         void* out, moe_dtype out_dt, void* workspace, size_t workspace_bytes,
                         void* stream) {
  moe_status st = check_sizes(shape, T);
  if (st != MOE_OK) return st;
  if (out_dt != MOE_F32 && out_dt != MOE_BF16) return MOE_ERR_DTYPE;
  if (kind != MOE_WEIGHTS_BF16 && kind != MOE_WEIGHTS_E4M3 && kind != MOE_WEIGHTS_INT8)
    return MOE_ERR_DTYPE;
  if (T == 0) return MOE_OK;
  if (!x || !experts || !topk_idx || !topk_w || !out || !workspace || (bias && !w_router))
    return MOE_ERR_NULL;
  if ((shared != nullptr) != (shape->f_shared != 0)) return MOE_ERR_NULL;
  if ((st = check_weights(*experts, kind)) != MOE_OK) return st;
  if (shared && (st = check_weights(*shared, kind)) != MOE_OK) return st;
  if (!aligned(x, 16) || !aligned(w_router, 16) || !aligned(bias, 4) || !aligned(topk_idx, 4) ||
      !aligned(topk_w, 4) || !aligned(out, 16) || !aligned(workspace, kWorkspaceAlign))
    return MOE_ERR_ALIGN;
  if (workspace_bytes < moe_layer_few_workspace_bytes(shape, T)) return MOE_ERR_WORKSPACE;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  moe::FewLayer g{};
  g.T = T;
  g.k = shape->top_k;
  g.d = shape->d;
  g.f = shape->f;
  g.E = shape->n_experts;
  g.shared = shared ? 1 : 0;
  g.x = x;
  g.topk_idx = topk_idx;
  g.topk_w = topk_w;
  g.gate_up = experts->gate_up;
  g.down = experts->down;
  g.gate_up_scales = experts->gate_up_scales;
  g.down_scales = experts->down_scales;
  if (shared) {
    g.shared_gate_up = shared->gate_up;
    g.shared_down = shared->down;
    g.shared_gate_up_scales = shared->gate_up_scales;
    g.shared_down_scales = shared->down_scales;
  }
  uint8_t* scratch = static_cast<uint8_t*>(workspace) + moe_route_workspace_bytes(shape, T);
  g.table = scratch;
  g.h = reinterpret_cast<uint16_t*>(scratch + scratch_of(shape, T).h);
  g.parts = reinterpret_cast<float*>(scratch + scratch_of(shape, T).parts);
  g.h_apart = static_cast<int64_t>(T) * (g.k + g.shared) * g.f;
  g.out = out;
  g.out_f32 = out_dt == MOE_F32;
  if (w_router) {
    const hipError_t e =
        moe::launch_route(T, g.d, g.E, g.k, x, true, w_router, bias,
                          static_cast<double*>(workspace), topk_idx, topk_w, s);
    if (e != hipSuccess) return hip_status(e);
  }
  return hip_status(moe::launch_layer_few(g,
                                          kind == MOE_WEIGHTS_BF16   ? moe::kFewBf16
                                          : kind == MOE_WEIGHTS_E4M3 ? moe::kFewE4m3
                                                                     : moe::kFewInt8,
                                          s));
}

}  // extern "C"
