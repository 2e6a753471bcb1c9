// Argument checks shared by C-ABI entry points in more than one source file.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "moe_int4.h"

namespace moe {

constexpr size_t kWorkspaceAlign = 256;

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline size_t round_up(size_t n) {
  return (n + kWorkspaceAlign - 1) / kWorkspaceAlign * kWorkspaceAlign;
}

inline moe_status hip_status(hipError_t e) {
  if (e == hipSuccess) return MOE_OK;
  if (e == hipErrorNotSupported) return MOE_ERR_UNSUPPORTED;
  return MOE_ERR_HIP;
}

// moe_combine's checks of its shape, token count and types (api.cpp), which
// its gradient shares.
moe_status combine_check(const moe_shape* shape, int32_t T, moe_dtype y_dt, moe_dtype out_dt);

// Every argument check of moe_layer_decode except the workspace's (api.cpp):
// MOE_OK, or the status moe_layer_decode would return for these arguments.
moe_status layer_decode_check(const moe_shape* shape, int32_t T, const void* x, moe_dtype x_dt,
                              const float* w_router, const float* bias, const uint8_t* experts,
                              const uint8_t* shared, const int32_t* topk_idx,
                              const float* topk_w, const int32_t* counts,
                              const int32_t* offsets, const int32_t* perm,
                              const int32_t* inv_perm, const int32_t* active,
                              const int32_t* n_active, const void* y, const void* y_shared,
                              const void* out, moe_dtype out_dt);

}  // namespace moe
