// The two norms and the residual around a block, in one pass over the row:
//   yh = y * a,  a = 1 / sqrt(mean(y^2) + eps)      (yh = y without w_post)
//   r  = res + scale * gate * (w_post * yh)
//   n  = w_pre * r * b,  b = 1 / sqrt(mean(r^2) + eps)
// and its gradient.  All of it is bound by memory: a row is read once into
// registers (8 columns per thread, d <= 8192), both statistics come from
// them in float32, and n is taken from r before r is rounded to its own type.
// One row of 6144 takes 4.2 us (launch and two meetings of the workgroup), 2048
// of bf16 (101 MB) 29 us, of float32 46; the gradient of 2048 rows of bf16 (151
// MB) 38 us for the rows, 4.0 TB/s, and 5 for the columns' sums, of float32 75 in
// all.
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

// v of the lane that DPP control CTRL names, inside rows of 16 lanes.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
      0, static_cast<int>(__float_as_uint(v)), CTRL, 0xF, 0xF, false)));
}
// Sum over each row of 16 lanes (quad_perm [1,0,3,2] and [2,3,0,1],
// row_half_mirror, row_mirror), every lane receiving it.
__device__ __forceinline__ float row_sum(float v) {
  v += dpp<0xB1>(v);
  v += dpp<0x4E>(v);
  v += dpp<0x141>(v);
  v += dpp<0x140>(v);
  return v;
}
__device__ __forceinline__ float readlane(float v, int lane) {
  return __uint_as_float(static_cast<uint32_t>(
      __builtin_amdgcn_readlane(static_cast<int>(__float_as_uint(v)), lane)));
}

// Sums of N values over the workgroup, in a fixed order (lanes and wavefronts
// by DPP: the shuffles through LDS that this replaced were a third of the
// gradient's time); sh: N x kMaxWaves floats not used since the last barrier.
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float (*sh)[kMaxWaves]) {
  const int waves = blockDim.x / kWave, lane = threadIdx.x % kWave;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = row_sum(v[i]);
    v[i] = (readlane(v[i], 0) + readlane(v[i], 16)) + (readlane(v[i], 32) + readlane(v[i], 48));
  }
  if (waves == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) sh[i][threadIdx.x / kWave] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = readlane(row_sum(lane < waves ? sh[i][lane & 15] : 0.0f), 0);
}
__device__ __forceinline__ float block_sum(float v, float (*sh)[kMaxWaves]) {
  float one[1] = {v};
  block_sums(one, sh);
  return one[0];
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
  for (int64_t row = blockIdx.x; row < g.T; row += gridDim.x) {
    const int64_t at = row * g.d + c;
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
        const float a = inv_rms(block_sum(sum_sq(y), &sh[0]), g.d, g.eps);
#pragma unroll
        for (int j = 0; j < kV; ++j) y[j] = w1[j] * (y[j] * a);
      }
#pragma unroll
      for (int j = 0; j < kV; ++j) r[j] = fmaf(g.scale * gt[j], y[j], r[j]);
    }
    if (in && g.res_out) store8(g.res_out, g.res_bf16, at, r);
    if (g.w_pre) {
      const float b = inv_rms(block_sum(in ? sum_sq(r) : 0.0f, &sh[1]), g.d, g.eps);
#pragma unroll
      for (int j = 0; j < kV; ++j) r[j] = w2[j] * (r[j] * b);
      if (in) store8(g.normed, g.normed_bf16, at, r);
    }
    if (gridDim.x < g.T) __syncthreads();  // the sums' scratch is free for the next row
  }
}

// 8 values of a row as they lie in memory.
struct Raw {
  uint4 lo, hi;  // hi: the second half of 8 float32
};
template <bool ALL_BF16>
__device__ __forceinline__ Raw raw8(const void* p, bool bf16, int64_t i) {
  Raw r{};
  if (ALL_BF16 || bf16) {
    r.lo = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
  } else {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
    r.lo = q[0];
    r.hi = q[1];
  }
  return r;
}
template <bool ALL_BF16>
__device__ __forceinline__ void values(const Raw& r, bool bf16, float (&v)[kV]) {
  const uint32_t w[8] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w, r.hi.x, r.hi.y, r.hi.z, r.hi.w};
  if (ALL_BF16 || bf16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kV; ++j) v[j] = __uint_as_float(w[j]);
  }
}

// One workgroup takes rows blockIdx.x, + gridDim.x, ...; the columns' sums
//   s1 = sum_t [gate_t] t ∘ yh      (dw_post, dgate of a broadcast gate)
//   s2 = sum_t dn ∘ rh              (dw_pre)
// stay in its registers and go to part[workgroup][2][d].  The gradient:
//   t  = dr + b (v - rh mean(v rh)),  v = w_pre dn, rh = r b     -> dres
//   dp = scale gate t;  dgate = scale t w_post yh
//   dy = a (q' - yh mean(q' yh)),     q' = w_post dp
// mean(q' yh) is linear in t, so with q = scale gate w_post yh it follows from
// the sums of q dr, q v and q r: after a, one round of five sums (with r^2 and
// v r) gives every scalar of the row, and a row costs two meetings of the
// workgroup.  With all-bf16 rows the next row is fetched before this row's
// sums (a row of float32 would not fit the registers twice).
// THREADS, the most of a launch, sets the registers a thread may hold (256, 168,
// 128): the widest rows have the fewest, and past 6144 columns some of a row goes
// through scratch (bf16 with a gate per token 20 bytes a lane, other types 44, 128
// with a gate per token; bf16 rows of 8192 none): 2048 x 8192 takes 48-58 us of
// bf16 (201 MB), 102 with a float32 residual (302 MB), 120 of float32 (403 MB).
// PER_TOKEN: a gate of T rows.
template <int THREADS, bool ALL_BF16, bool PER_TOKEN>
__global__ __launch_bounds__(THREADS) void norm_grad_rows(BlockNorm g) {
  __shared__ float sh[2][6][kMaxWaves];  // by the row's parity
  const int c = threadIdx.x * kV;
  const bool in = c < g.d;
  float w1[kV], w2[kV], gt[kV], s1[kV] = {}, s2[kV] = {};
  ones(w1);
  ones(w2);
  ones(gt);
  if (in) {
    if (g.w_post) load8(g.w_post, false, c, w1);
    if (g.w_pre) load8(g.w_pre, false, c, w2);
    if (!PER_TOKEN && g.gate) load8(g.gate, g.y_bf16, c, gt);
  }
  const float inv_d = 1.0f / static_cast<float>(g.d);
  Raw ry{}, rr{}, rt{}, rn{}, rg{};
  auto read = [&](int64_t row) {
    const int64_t at = row * g.d + c;
    if (!in || row >= g.T) return;
    if (g.y) ry = raw8<ALL_BF16>(g.y, g.y_bf16, at);
    if (g.res) rr = raw8<ALL_BF16>(g.res, g.res_bf16, at);
    if (g.dr) rt = raw8<ALL_BF16>(g.dr, g.res_bf16, at);
    if (g.w_pre) rn = raw8<ALL_BF16>(g.dn, g.normed_bf16, at);
    if (PER_TOKEN) rg = raw8<ALL_BF16>(g.gate, g.y_bf16, at);
  };
  read(blockIdx.x);
  int odd = 0;
  for (int64_t row = blockIdx.x; row < g.T; row += gridDim.x, odd ^= 1) {
    const int64_t at = row * g.d + c;
    float y[kV], r[kV], t[kV], dn[kV];
    values<ALL_BF16>(ry, g.y_bf16, y);
    values<ALL_BF16>(rr, g.res_bf16, r);
    values<ALL_BF16>(rt, g.res_bf16, t);
    values<ALL_BF16>(rn, g.normed_bf16, dn);
    if (PER_TOKEN) values<ALL_BF16>(rg, g.y_bf16, gt);
    if (ALL_BF16) read(row + gridDim.x);
    float a = 1.0f;
    if (g.y && g.w_post) {
      a = inv_rms(block_sum(sum_sq(y), &sh[odd][5]), g.d, g.eps);
#pragma unroll
      for (int j = 0; j < kV; ++j) y[j] *= a;  // yh
    }
    float sum[5] = {};  // r^2, v r, q dr, q v, q r
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const float q = g.scale * gt[j] * (w1[j] * y[j]);
      const float v = w2[j] * dn[j];
      if (g.y) r[j] += q;
      sum[0] = fmaf(r[j], r[j], sum[0]);
      sum[1] = fmaf(v, r[j], sum[1]);
      sum[2] = fmaf(q, t[j], sum[2]);
      sum[3] = fmaf(q, v, sum[3]);
      sum[4] = fmaf(q, r[j], sum[4]);
    }
    block_sums(sum, sh[odd]);
    float mean_qt = sum[2];
    if (g.w_pre) {
      const float b = inv_rms(sum[0], g.d, g.eps);
      const float m = b * b * sum[1] * inv_d;  // mean(v rh) b, so t = dr + b (v - m r)
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        s2[j] = fmaf(dn[j], r[j] * b, s2[j]);
        t[j] = fmaf(b, fmaf(-m, r[j], w2[j] * dn[j]), t[j]);
      }
      mean_qt = fmaf(b, fmaf(-m, sum[4], sum[3]), mean_qt);
    }
    mean_qt *= inv_d;  // mean(q' yh)
    if (in && g.dres) store8(g.dres, g.res_bf16, at, t);
    if (g.y) {
      if (PER_TOKEN && in && g.dgate) {
        float dg[kV];
#pragma unroll
        for (int j = 0; j < kV; ++j) dg[j] = g.scale * t[j] * (w1[j] * y[j]);
        store8(g.dgate, g.y_bf16, at, dg);
      }
      float dp[kV];
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        s1[j] = fmaf(PER_TOKEN ? t[j] * gt[j] : t[j], y[j], s1[j]);
        dp[j] = g.scale * (t[j] * gt[j]) * w1[j];
        if (g.w_post) dp[j] = a * fmaf(-mean_qt, y[j], dp[j]);
      }
      if (in && g.dy) store8(g.dy, g.y_bf16, at, dp);
    }
    if (!ALL_BF16) read(row + gridDim.x);
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
#pragma unroll 8
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
  // no rows: zeros, also where the gate or w_post is not finite
  const float scale = parts > 0 ? g.scale : 0.0f;
  float gate = 1.0f;
  if (cast && parts > 0)
    gate = g.y_bf16 ? bf16_to_f32(static_cast<const uint16_t*>(g.gate)[c])
                    : static_cast<const float*>(g.gate)[c];
  if (g.dw_post) g.dw_post[c] = scale * gate * s1;
  if (g.dw_pre) g.dw_pre[c] = s2;
  if (cast && g.dgate) {
    const float v = scale * (g.w_post && parts > 0 ? g.w_post[c] : 1.0f) * s1;
    if (g.y_bf16)
      static_cast<uint16_t*>(g.dgate)[c] = f32_to_bf16(v);
    else
      static_cast<float*>(g.dgate)[c] = v;
  }
}

dim3 row_block(int d) { return dim3((d / kV + kWave - 1) / kWave * kWave); }

}  // namespace

// Workgroups of the gradient: one per CU, more where a row takes less than 16
// wavefronts' share of it, and no more than rows.
int norm_grad_parts(int T, int d) {
  const int waves = (d / kV + kWave - 1) / kWave;
  const int parts = 256 * (waves > 8 ? 1 : waves > 4 ? 2 : 4);
  return T < parts ? T : parts;
}

template <int THREADS>
hipError_t launch_norm_grad_rows(const BlockNorm& g, int parts, hipStream_t stream) {
  // by the operands there are: a type given for one that is absent says nothing
  // (2048 x 6144 without a pre norm, whose type the binding gives as float32: 42
  // us by the kernel for mixed rows, 37 by the one for bf16; 2048 x 8192 58 and 41)
  const bool all_bf16 = (!g.y || g.y_bf16) && ((!g.res && !g.dr && !g.dres) || g.res_bf16) &&
                        (!g.w_pre || g.normed_bf16);
  const bool per_token = g.gate && g.gate_rows != 1;
  auto go = [&](auto kernel) { return launch(kernel, dim3(parts), row_block(g.d), 0, stream, g); };
  if (all_bf16)
    return per_token ? go(norm_grad_rows<THREADS, true, true>)
                     : go(norm_grad_rows<THREADS, true, false>);
  return per_token ? go(norm_grad_rows<THREADS, false, true>)
                   : go(norm_grad_rows<THREADS, false, false>);
}

hipError_t launch_block_norm(const BlockNorm& g, hipStream_t stream) {
  // a grid holds fewer than 2^32 threads
  constexpr int kMaxGrid = 1 << 21;
  return launch(norm_rows, dim3(g.T < kMaxGrid ? g.T : kMaxGrid), row_block(g.d), 0, stream, g);
}

hipError_t launch_block_norm_grad(const BlockNorm& g, hipStream_t stream) {
  const int parts = norm_grad_parts(g.T, g.d);
  if (parts > 0) {
    const uint32_t threads = row_block(g.d).x;
    const hipError_t e = threads <= 512   ? launch_norm_grad_rows<512>(g, parts, stream)
                         : threads <= 768 ? launch_norm_grad_rows<768>(g, parts, stream)
                                          : launch_norm_grad_rows<1024>(g, parts, stream);
    if (e != hipSuccess || !g.columns) return e;
  }
  return launch(norm_grad_columns, dim3((g.d + kWave - 1) / kWave), dim3(1024), 0, stream, g,
                parts);
}

}  // namespace moe
