// The two norms and the residual around a block, in one pass over the row:
//   yh = y * a,  a = 1 / sqrt(mean(y^2) + eps)      (yh = y without w_post)
//   r  = res + scale * gate * (w_post * yh)
//   n  = w_pre * r * b,  b = 1 / sqrt(mean(r^2) + eps)
// and its gradient.  All of it is bound by memory: a row is read once into
// registers (8 columns per thread, d <= 8192), both statistics come from
// them in float32, and n is taken from r before r is rounded to its own type.
#include "common.h"
#include "launch.h"

#pragma clang fp contract(off)  // the fused multiply-adds are written out

namespace moe {

namespace {

constexpr int kV = 8;
constexpr int kMaxWaves = 16;  // 1024 threads x 8 columns

__device__ __forceinline__ void load8(const void* p, bool bf16, int64_t i, float (&v)[kV]) {
  if (bf16) {
    const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  } else {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

__device__ __forceinline__ void store8(void* p, bool bf16, int64_t i, const float (&v)[kV]) {
  if (bf16) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = static_cast<uint32_t>(f32_to_bf16(v[2 * j])) |
             (static_cast<uint32_t>(f32_to_bf16(v[2 * j + 1])) << 16);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    float* o = static_cast<float*>(p) + i;
    *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(o + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// Sum over the workgroup in a fixed order; sh: kMaxWaves floats not used
// since the last barrier.
__device__ __forceinline__ float block_sum(float v, float* sh) {
  v = group_sum(v, kWave);
  const int waves = blockDim.x / kWave;
  if (waves == 1) return v;
  if (threadIdx.x % kWave == 0) sh[threadIdx.x / kWave] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < waves; ++w) s += sh[w];
  return s;
}

__device__ __forceinline__ float sum_sq(const float (&v)[kV]) {
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < kV; ++j) s = fmaf(v[j], v[j], s);
  return s;
}

__device__ __forceinline__ void ones(float (&v)[kV]) {
#pragma unroll
  for (int j = 0; j < kV; ++j) v[j] = 1.0f;
}

__device__ __forceinline__ float inv_rms(float sq, int d, float eps) {
  return 1.0f / sqrtf(sq / static_cast<float>(d) + eps);
}

__global__ __launch_bounds__(1024) void norm_rows(BlockNorm g) {
  __shared__ float sh[2][kMaxWaves];
  const int c = threadIdx.x * kV;
  const bool in = c < g.d;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * g.d + c;
  float y[kV] = {}, r[kV] = {}, w1[kV] = {}, gt[kV], w2[kV] = {};
  ones(gt);
  if (in) {
    if (g.y) load8(g.y, g.y_bf16, at, y);
    if (g.res) load8(g.res, g.res_bf16, at, r);
    if (g.w_post) load8(g.w_post, false, c, w1);
    if (g.gate) load8(g.gate, g.y_bf16, g.gate_rows == 1 ? c : at, gt);
    if (g.w_pre) load8(g.w_pre, false, c, w2);
  }
  if (g.y) {
    if (g.w_post) {
      const float a = inv_rms(block_sum(sum_sq(y), sh[0]), g.d, g.eps);
#pragma unroll
      for (int j = 0; j < kV; ++j) y[j] = w1[j] * (y[j] * a);
    }
#pragma unroll
    for (int j = 0; j < kV; ++j) r[j] = fmaf(g.scale * gt[j], y[j], r[j]);
  }
  if (in && g.res_out) store8(g.res_out, g.res_bf16, at, r);
  if (g.w_pre) {
    const float b = inv_rms(block_sum(in ? sum_sq(r) : 0.0f, sh[1]), g.d, g.eps);
#pragma unroll
    for (int j = 0; j < kV; ++j) r[j] = w2[j] * (r[j] * b);
    if (in) store8(g.normed, g.normed_bf16, at, r);
  }
}

// One workgroup takes rows blockIdx.x, + gridDim.x, ...; the columns' sums
//   s1 = sum_t [gate_t] dr ∘ yh     (dw_post, dgate of a broadcast gate)
//   s2 = sum_t dn ∘ r b             (dw_pre)
// stay in its registers and go to part[workgroup][2][d].  The gradient:
//   t  = dr + b (v - rh mean(v rh)),  v = w_pre dn, rh = r b     -> dres
//   dp = scale gate t;  dgate = scale t w_post yh
//   dy = a (v - yh mean(v yh)),       v = w_post dp
__global__ __launch_bounds__(1024) void norm_grad_rows(BlockNorm g) {
  __shared__ float sh[4][kMaxWaves];
  const int c = threadIdx.x * kV;
  const bool in = c < g.d;
  float w1[kV], w2[kV], g1[kV], s1[kV] = {}, s2[kV] = {};
  ones(w1);
  ones(w2);
  ones(g1);
  if (in) {
    if (g.w_post) load8(g.w_post, false, c, w1);
    if (g.w_pre) load8(g.w_pre, false, c, w2);
    if (g.gate && g.gate_rows == 1) load8(g.gate, g.y_bf16, c, g1);
  }
  const float inv_d = 1.0f / static_cast<float>(g.d);
  const bool per_token = g.gate && g.gate_rows != 1;
  for (int64_t row = blockIdx.x; row < g.T; row += gridDim.x) {
    const int64_t at = row * g.d + c;
    float y[kV] = {}, r[kV] = {}, t[kV] = {}, dn[kV] = {}, gt[kV];
#pragma unroll
    for (int j = 0; j < kV; ++j) gt[j] = g1[j];
    if (in) {
      if (g.y) load8(g.y, g.y_bf16, at, y);
      if (g.res) load8(g.res, g.res_bf16, at, r);
      if (per_token) load8(g.gate, g.y_bf16, at, gt);
      if (g.dr) load8(g.dr, g.res_bf16, at, t);
      if (g.w_pre) load8(g.dn, g.normed_bf16, at, dn);
    }
    float a = 1.0f;
    if (g.y && g.w_post) {
      a = inv_rms(block_sum(sum_sq(y), sh[0]), g.d, g.eps);
#pragma unroll
      for (int j = 0; j < kV; ++j) y[j] *= a;  // yh
    }
    if (g.y) {
#pragma unroll
      for (int j = 0; j < kV; ++j) r[j] = fmaf(g.scale * gt[j], w1[j] * y[j], r[j]);
    }
    if (g.w_pre) {
      const float b = inv_rms(block_sum(in ? sum_sq(r) : 0.0f, sh[1]), g.d, g.eps);
      float dot = 0.0f;
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        r[j] *= b;  // rh
        s2[j] = fmaf(dn[j], r[j], s2[j]);
        dn[j] *= w2[j];
        dot = fmaf(dn[j], r[j], dot);
      }
      const float mean = block_sum(in ? dot : 0.0f, sh[2]) * inv_d;
#pragma unroll
      for (int j = 0; j < kV; ++j) t[j] = fmaf(b, fmaf(-mean, r[j], dn[j]), t[j]);
    }
    if (in && g.dres) store8(g.dres, g.res_bf16, at, t);
    if (g.y) {
      if (per_token) {
        float dg[kV];
#pragma unroll
        for (int j = 0; j < kV; ++j) dg[j] = g.scale * t[j] * (w1[j] * y[j]);
        if (in && g.dgate) store8(g.dgate, g.y_bf16, at, dg);
#pragma unroll
        for (int j = 0; j < kV; ++j) t[j] *= gt[j];
      }
      float dot = 0.0f, dp[kV];
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        s1[j] = fmaf(t[j], y[j], s1[j]);
        dp[j] = g.scale * (per_token ? t[j] : t[j] * gt[j]) * w1[j];
        dot = fmaf(dp[j], y[j], dot);
      }
      if (g.w_post) {
        const float mean = block_sum(in ? dot : 0.0f, sh[3]) * inv_d;
#pragma unroll
        for (int j = 0; j < kV; ++j) dp[j] = a * fmaf(-mean, y[j], dp[j]);
      }
      if (in && g.dy) store8(g.dy, g.y_bf16, at, dp);
    }
    __syncthreads();  // the sums' scratch is free for the next row
  }
  if (in && g.part) {
    const int64_t o = static_cast<int64_t>(blockIdx.x) * 2 * g.d + c;
    store8(g.part, false, o, s1);
    store8(g.part, false, o + g.d, s2);
  }
}

// The columns' sums over the workgroups, in order: 64 columns per workgroup,
// 16 wavefronts each adding every 16th partial, then those 16.
__global__ __launch_bounds__(1024) void norm_grad_columns(BlockNorm g, int parts) {
  __shared__ float sh[2][kMaxWaves][kWave];
  const int lane = threadIdx.x % kWave, wv = threadIdx.x / kWave;
  const int c = blockIdx.x * kWave + lane;
  float s1 = 0.0f, s2 = 0.0f;
  if (c < g.d)
    for (int p = wv; p < parts; p += kMaxWaves) {
      const float* row = g.part + static_cast<int64_t>(p) * 2 * g.d;
      s1 += row[c];
      s2 += row[g.d + c];
    }
  sh[0][wv][lane] = s1;
  sh[1][wv][lane] = s2;
  __syncthreads();
  if (wv != 0 || c >= g.d) return;
  s1 = s2 = 0.0f;
  for (int w = 0; w < kMaxWaves; ++w) {
    s1 += sh[0][w][lane];
    s2 += sh[1][w][lane];
  }
  const bool cast = g.gate && g.gate_rows == 1;
  float gate = 1.0f;
  if (cast)
    gate = g.y_bf16 ? bf16_to_f32(static_cast<const uint16_t*>(g.gate)[c])
                    : static_cast<const float*>(g.gate)[c];
  if (g.dw_post) g.dw_post[c] = g.scale * gate * s1;
  if (g.dw_pre) g.dw_pre[c] = s2;
  if (cast && g.dgate) {
    const float v = g.scale * (g.w_post ? g.w_post[c] : 1.0f) * s1;
    if (g.y_bf16)
      static_cast<uint16_t*>(g.dgate)[c] = f32_to_bf16(v);
    else
      static_cast<float*>(g.dgate)[c] = v;
  }
}

dim3 row_block(int d) { return dim3((d / kV + kWave - 1) / kWave * kWave); }

}  // namespace

int norm_grad_parts(int T) { return T < 512 ? T : 512; }

hipError_t launch_block_norm(const BlockNorm& g, hipStream_t stream) {
  return launch(norm_rows, dim3(g.T), row_block(g.d), 0, stream, g);
}

hipError_t launch_block_norm_grad(const BlockNorm& g, hipStream_t stream) {
  const int parts = norm_grad_parts(g.T);
  if (parts > 0) {
    const hipError_t e = launch(norm_grad_rows, dim3(parts), row_block(g.d), 0, stream, g);
    if (e != hipSuccess || !g.columns) return e;
  }
  return launch(norm_grad_columns, dim3((g.d + kWave - 1) / kWave), dim3(1024), 0, stream, g,
                parts);
}

}  // namespace moe
