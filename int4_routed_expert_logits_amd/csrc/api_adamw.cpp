// C ABI of include/moe_int4_adamw.h: like api.cpp, every argument is checked on
// the host, without a HIP call, before anything is enqueued.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "api_internal.h"
#include "launch.h"
#include "moe_int4_adamw.h"

namespace {

using moe::aligned;

constexpr int32_t kMaxTensors = 1 << 20;
constexpr int64_t kMaxElements = int64_t(1) << 40;

moe_status check_tensor(const moe_adamw_tensor& t) {
  if (t.n < 0) return MOE_ERR_SHAPE;
  if (t.n > kMaxElements) return MOE_ERR_UNSUPPORTED;
  if ((t.p_dt != MOE_F32 && t.p_dt != MOE_BF16) || (t.g_dt != MOE_F32 && t.g_dt != MOE_BF16) ||
      (t.master && t.p_dt != MOE_BF16))
    return MOE_ERR_DTYPE;
  if (t.n == 0) return MOE_OK;
  if (!t.p || !t.g || !t.m || !t.v || (t.m_scales != nullptr) != (t.v_scales != nullptr))
    return MOE_ERR_NULL;
  const size_t state = t.m_scales ? 1 : 4;
  if (!aligned(t.p, t.p_dt == MOE_F32 ? 4 : 2) || !aligned(t.master, 4) ||
      !aligned(t.g, t.g_dt == MOE_F32 ? 4 : 2) || !aligned(t.m, state) || !aligned(t.v, state) ||
      !aligned(t.m_scales, 4) || !aligned(t.v_scales, 4))
    return MOE_ERR_ALIGN;
  return MOE_OK;
}

moe::AdamWTensor get_tensor(const void* tensors, int i) {
  const moe_adamw_tensor& t = static_cast<const moe_adamw_tensor*>(tensors)[i];
  moe::AdamWTensor r{};
  r.n = t.n;
  r.p = t.p;
  r.master = t.master;
  r.g = t.g;
  r.m = t.m;
  r.v = t.v;
  r.m_scales = t.m_scales;
  r.v_scales = t.v_scales;
  r.p_bf16 = t.p_dt == MOE_BF16;
  r.g_bf16 = t.g_dt == MOE_BF16;
  const size_t state = t.m_scales ? 4 : 16;
  r.wide = aligned(t.p, r.p_bf16 ? 8 : 16) && aligned(t.master, 16) &&
           aligned(t.g, r.g_bf16 ? 8 : 16) && aligned(t.m, state) && aligned(t.v, state);
  return r;
}

// Whether codes of moments go to the nearest (adamw.hip): v fast enough to fall by
// such codes, and 2 to 5 times slower than m (0.9 and 0.95 are just that, hence the
// room for their last places).
bool nearest_codes(double beta1, double beta2) {
  const double a = 1.0 - beta1, b = 1.0 - beta2, room = 1.0 + 1e-9;
  return beta2 <= 0.95 && 2.0 * b <= a * room && a <= 5.0 * b * room;
}

bool at_least_zero(double v) { return isfinite(v) && v >= 0.0; }

}  // namespace

extern "C" {

moe_status moe_adamw(const moe_adamw_tensor* tensors, int32_t n_tensors, const int64_t* step,
                     double lr, double beta1, double beta2, double eps, double weight_decay,
                     const float* grad_scale, void* stream) {
  if (n_tensors < 0) return MOE_ERR_SHAPE;
  if (n_tensors > kMaxTensors) return MOE_ERR_UNSUPPORTED;
  if (!at_least_zero(lr) || !at_least_zero(weight_decay) || !at_least_zero(beta1) || beta1 >= 1.0 ||
      !at_least_zero(beta2) || beta2 >= 1.0 || !at_least_zero(eps) ||
      !isfinite(static_cast<float>(eps)) || !(static_cast<float>(eps) > 0.0f) ||
      !isfinite(static_cast<float>(lr)) || !isfinite(static_cast<float>(1.0 - lr * weight_decay)))
    return MOE_ERR_SHAPE;
  if (n_tensors > 0 && !tensors) return MOE_ERR_NULL;
  bool any = false;
  for (int32_t i = 0; i < n_tensors; ++i) {
    const moe_status st = check_tensor(tensors[i]);
    if (st != MOE_OK) return st;
    any = any || tensors[i].n > 0;
  }
  if (!any) return MOE_OK;
  if (!step) return MOE_ERR_NULL;
  if (!aligned(step, 8) || !aligned(grad_scale, 4)) return MOE_ERR_ALIGN;
  moe::AdamWStep s{};
  s.step = step;
  s.grad_scale = grad_scale;
  s.lr = lr;
  s.log_beta1 = log(beta1);  // -inf for 0: a power of 0
  s.log_beta2 = log(beta2);
  s.beta1 = static_cast<float>(beta1);
  s.rest1 = static_cast<float>(1.0 - beta1);
  s.beta2 = static_cast<float>(beta2);
  s.rest2 = static_cast<float>(1.0 - beta2);
  s.eps = static_cast<float>(eps);
  s.keep = static_cast<float>(1.0 - lr * weight_decay);
  s.nearest = nearest_codes(beta1, beta2);
  return moe::hip_status(moe::launch_adamw(moe::AdamWSource{tensors, get_tensor}, n_tensors, s,
                                           static_cast<hipStream_t>(stream)));
}

}  // extern "C"
