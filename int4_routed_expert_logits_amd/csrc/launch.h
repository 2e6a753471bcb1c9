// Internal host-side launchers, one per kernel family.  Arguments have been
// validated by the C-ABI layer (api.cpp) before any of these is called; each
// returns the hipError_t of its launches.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <tuple>
#include <utility>

namespace moe {

// Launch through hipLaunchKernel so the launch status comes back directly,
// without touching the thread's sticky last-error state.
template <typename... KArgs, typename... Args>
hipError_t launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t shmem,
                  hipStream_t stream, Args&&... args) {
  std::tuple<KArgs...> held(static_cast<KArgs>(std::forward<Args>(args))...);
  return std::apply(
      [&](auto&... a) {
        void* ptrs[] = {static_cast<void*>(&a)...};
        return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, ptrs, shmem,
                               stream);
      },
      held);
}

// route.hip: float64 logits then top-k + renormalised softmax.  The
// workspace holds float64 logits, split into route_parts() partial sums per
// (token, expert) and part of d.
int route_parts(int T, int d, int E);
size_t route_workspace(int T, int d, int E);
hipError_t launch_route(int T, int d, int E, int k, const void* x, bool x_bf16,
                        const float* w_router, const float* bias, double* logits,
                        int32_t* topk_idx, float* topk_w, hipStream_t stream);

// union.hip: batch-union grouping in one workgroup.
hipError_t launch_union(int n_slots, int E, const int32_t* topk_idx, int32_t* counts,
                        int32_t* offsets, int32_t* perm, int32_t* inv_perm, int32_t* active,
                        int32_t* n_active, hipStream_t stream);

// The batch-union outputs (moe_union's arrays).
struct UnionOut {
  int32_t *counts, *offsets, *perm, *inv_perm, *active, *n_active;
};

// route.hip: the router and the batch-union of its result; small batches run
// top-k and union in one kernel, the rest as launch_route + launch_union.
hipError_t launch_route_union(int T, int d, int E, int k, const void* x, bool x_bf16,
                              const float* w_router, const float* bias, double* logits,
                              int32_t* topk_idx, float* topk_w, const UnionOut& u,
                              hipStream_t stream);

// route.hip: only the float64 logit partial sums of launch_route (the
// workspace's [T][E][route_parts()] doubles).
hipError_t launch_router_logits(int T, int d, int E, const void* x, bool x_bf16,
                                const float* w_router, double* part, hipStream_t stream);

// quant.hip: float weights -> int4 codes + float16 scales (per 64-column
// group, or per row).
hipError_t launch_quantize(int N, int K, const void* w, bool f32, bool per_row, uint8_t* codes,
                           void* scales, hipStream_t stream);

struct FfnProblem {
  int T, d, f, E, k;
  bool has_shared;
  bool x_bf16;
  bool mxfp4 = false;  // MXFP4 blocks instead of int4 gs64
  size_t block_bytes;
  const void* x;
  const uint8_t* experts;
  const uint8_t* shared;
  const int32_t* offsets;
  const int32_t* perm;
  const int32_t* active;
  const int32_t* n_active;
  void* y;
  void* y_shared;
  void* workspace;
};

// ffn_decode.hip: int4 GEMV, float32 intermediate and outputs.
size_t ffn_decode_workspace(int T, int k, int E, int d, int f, bool has_shared);
hipError_t launch_ffn_decode(const FfnProblem& p, hipStream_t stream);

// ffn_decode.hip: the same FFN for a small batch whose top-k and grouping
// the gate/up kernel derives itself from the router's partial sums (part,
// P parts per logit), writing them to topk_idx / topk_w and u (p.offsets,
// p.perm, p.active and p.n_active must be u's arrays).
struct RouteGroup {
  const double* part;
  int P;
  const float* bias;
  int32_t* topk_idx;
  float* topk_w;
  UnionOut u;
};
// Whether launch_ffn_decode_grouping takes this problem (batch size, experts,
// parts per logit, LDS).
bool ffn_decode_groups_batch(const FfnProblem& p, int P);
hipError_t launch_ffn_decode_grouping(const FfnProblem& p, const RouteGroup& rg,
                                      hipStream_t stream);

// ffn_prefill.hip: grouped GEMM on bf16 MFMA, bf16 intermediate and outputs.
size_t ffn_prefill_workspace(int T, int k, int E, int d, int f, bool has_shared);
hipError_t launch_ffn_prefill(const FfnProblem& p, hipStream_t stream);

// pack.hip: canonical -> packed expert blocks (int4 gs64, or MXFP4).
hipError_t launch_pack(int d, int f, long long n_blocks, size_t block_bytes, const uint8_t* src,
                       uint8_t* dst, hipStream_t stream);
hipError_t launch_pack_mxfp4(int d, int f, long long n_blocks, size_t block_bytes,
                             const uint8_t* src, uint8_t* dst, hipStream_t stream);

// combine.hip
hipError_t launch_combine(int T, int d, int k, const void* y, const void* y_shared, bool y_bf16,
                          const int32_t* inv_perm, const float* topk_w, void* out,
                          bool out_bf16, hipStream_t stream);

// grouped_mm.hip: products over rows grouped by expert.
struct GroupedMm {
  const uint8_t* r;  // operand indexed by the output's row: x or its codes, dy
  const uint8_t* f;  // ... by the output's column: w or its codes, x
  const float *r_scale, *f_scale;  // kGroupedCodes: per (row, 128 columns), per 128 x 128
  const int32_t* offsets;          // [E + 1]
  const int32_t* rows;             // [P] source rows of x times div, or NULL
  uint32_t row_limit, div_magic;   // rows entries below row_limit are valid
  void* out;
  void* workspace;
  int E, P, N, K;
  int split;  // kGroupedWeights: parts of a group's rows, joined through workspace
  bool out_f32;
};
size_t grouped_dw_workspace(int E, int P, int N, int K);
enum GroupedKind { kGroupedRows, kGroupedInput, kGroupedWeights, kGroupedCodes };
hipError_t launch_grouped_mm(const GroupedMm& g, GroupedKind kind, hipStream_t stream);

// blockscale.hip: e4m3 codes with a float32 scale per 128 columns (or per 128
// x 128), and SwiGLU over grouped rows (scales: h holds codes).
hipError_t launch_blockscale_quantize(int n_mats, int R, int K, const void* x, bool f32,
                                      bool square, uint8_t* codes, float* scales,
                                      hipStream_t stream);
hipError_t launch_swiglu(int P, int f, const void* gu, bool f32, void* h, float* scales,
                         const int32_t* n_rows, hipStream_t stream);
hipError_t launch_swiglu_grad(int P, int f, const void* gu, const void* dh, bool f32, void* dgu,
                              const int32_t* n_rows, hipStream_t stream);

// block_norm.hip: the norms and the residual around a block, and the gradient.
struct BlockNorm {
  int T, d, gate_rows;
  float scale, eps;
  bool y_bf16, res_bf16, normed_bf16;
  const void *y, *res, *gate;
  const float *w_post, *w_pre;
  void *res_out, *normed;                 // forward
  const void *dr, *dn;                    // gradient: of res_out, of normed
  void *dy, *dres, *dgate;
  float *dw_post, *dw_pre, *part;         // part: [norm_grad_parts][2][d]
  bool columns;                           // a sum over the rows is asked for
};
int norm_grad_parts(int T, int d);
hipError_t launch_block_norm(const BlockNorm& g, hipStream_t stream);
hipError_t launch_block_norm_grad(const BlockNorm& g, hipStream_t stream);

// combine.hip: gradient of launch_combine.
hipError_t launch_combine_grad(int T, int d, int k, const void* dout, bool out_bf16,
                               const void* y, bool y_bf16, const int32_t* inv_perm,
                               const float* topk_w, void* dy, float* dtopk_w, hipStream_t stream);

}  // namespace moe
