// 8-bit floats with a scale per block of 128: rows (1 x 128, activations) or
// 128 x 128 (weights) to e4m3 codes and float32 scales, and SwiGLU over
// grouped rows (also straight to codes) with its gradient.
//
// The scale is a power of two, the smallest that keeps the block's largest
// magnitude within 448 (e4m3's largest): dividing by it is exact, so every
// code is the value rounded once, and no rounding of a quotient can move it.
// e4m3 is a floating format, so a scale that is not exactly absmax / 448 costs
// no precision outside its subnormals.
#include "common.h"
#include "launch.h"

#pragma clang fp contract(off)  // the fused multiply-adds are written out

namespace moe {

namespace {

constexpr int kV = 8;         // columns per thread
constexpr int kBlock = 128;   // columns per scale
constexpr int kGroupLanes = kBlock / kV;
constexpr int kThreads = 256;

template <bool F32>
__device__ __forceinline__ void load8(const void* p, size_t i, float (&v)[kV]) {
  if constexpr (F32) {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
}

template <bool F32>
__device__ __forceinline__ void store8(void* p, size_t i, const float (&v)[kV]) {
  if constexpr (F32) {
    float* o = static_cast<float*>(p) + i;
    *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(o + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = static_cast<uint32_t>(f32_to_bf16(v[2 * j])) |
             (static_cast<uint32_t>(f32_to_bf16(v[2 * j + 1])) << 16);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

__device__ __forceinline__ bool finite(float v) {
  return (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u;
}

// Largest finite magnitude of 8 values.
__device__ __forceinline__ float absmax8(const float (&v)[kV]) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < kV; ++j) m = fmaxf(m, finite(v[j]) ? fabsf(v[j]) : 0.0f);
  return m;
}

// Exponent n of the block's scale 2^n: the smallest n >= -126 with
// absmax <= 448 * 2^n (448 = 1.75 * 2^8); 0 for a block of zeros.
__device__ __forceinline__ int scale_exponent(float absmax) {
  const uint32_t b = __float_as_uint(absmax);
  if (b == 0u) return 0;
  const int e = static_cast<int>(b >> 23) - 127;
  return max(-126, (b & 0x7FFFFFu) <= 0x600000u ? e - 8 : e - 7);
}
__device__ __forceinline__ float two_to(int n) {
  return __uint_as_float(static_cast<uint32_t>(n + 127) << 23);
}

// 8 codes of v * 2^-n, round to nearest even (the hardware conversion); a
// non-finite value gives a NaN code.
__device__ __forceinline__ uint2 codes8(const float (&v)[kV], int n) {
  const float inv = two_to(-n);
  float q[kV];
#pragma unroll
  for (int j = 0; j < kV; ++j) q[j] = finite(v[j]) ? v[j] * inv : __uint_as_float(0x7FC00000u);
  uint2 r;
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
  r.x = static_cast<uint32_t>(lo);
  r.y = static_cast<uint32_t>(hi);
  return r;
}

__device__ __forceinline__ float group_max(float m) {
  for (int off = kGroupLanes / 2; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, kWave));
  return m;
}

// Rows: 16 lanes hold a block of 128 columns.
template <bool F32>
__global__ __launch_bounds__(kThreads) void quant_rows(int64_t blocks, int K, int KB,
                                                       const void* __restrict__ x,
                                                       uint8_t* __restrict__ codes,
                                                       float* __restrict__ scales) {
  const int64_t b = static_cast<int64_t>(blockIdx.x) * (kThreads / kGroupLanes) +
                    threadIdx.x / kGroupLanes;
  if (b >= blocks) return;
  const int64_t row = b / KB;
  const int c = static_cast<int>(b - row * KB) * kBlock + (threadIdx.x % kGroupLanes) * kV;
  float v[kV] = {};
  if (c < K) load8<F32>(x, row * K + c, v);
  const int n = scale_exponent(group_max(absmax8(v)));
  if (c < K) *reinterpret_cast<uint2*>(codes + row * K + c) = codes8(v, n);
  if (threadIdx.x % kGroupLanes == 0) scales[b] = two_to(n);
}

// 128 x 128: one workgroup per block, 8 rows of 8 columns per thread.
template <bool F32>
__global__ __launch_bounds__(kThreads) void quant_blocks(int R, int K, int RB, int KB,
                                                         const void* __restrict__ x,
                                                         uint8_t* __restrict__ codes,
                                                         float* __restrict__ scales) {
  __shared__ float sh[kThreads / kWave];
  constexpr int kRows = kThreads / kGroupLanes;  // rows per pass
  const int64_t b = blockIdx.x;
  const int kb = static_cast<int>(b % KB), rb = static_cast<int>((b / KB) % RB);
  const int64_t base = (b / KB / RB) * R;  // first row of the matrix
  const int c = kb * kBlock + (threadIdx.x % kGroupLanes) * kV;
  const int r0 = rb * kBlock + threadIdx.x / kGroupLanes;
  float v[kBlock / kRows][kV] = {};
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < kBlock / kRows; ++i)
    if (c < K && r0 + i * kRows < R) {
      load8<F32>(x, (base + r0 + i * kRows) * K + c, v[i]);
      m = fmaxf(m, absmax8(v[i]));
    }
  for (int off = kWave / 2; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, kWave));
  if (threadIdx.x % kWave == 0) sh[threadIdx.x / kWave] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / kWave; ++w) m = fmaxf(m, sh[w]);
  const int n = scale_exponent(m);
#pragma unroll
  for (int i = 0; i < kBlock / kRows; ++i)
    if (c < K && r0 + i * kRows < R)
      *reinterpret_cast<uint2*>(codes + (base + r0 + i * kRows) * K + c) = codes8(v[i], n);
  if (threadIdx.x == 0) scales[b] = two_to(n);
}

// A thread's row and first column in a launch of `segs` workgroups per row
// group, 2^lg threads per row.
struct Spot {
  int64_t row;
  int c;
};
__device__ __forceinline__ Spot spot(int segs, int lg) {
  const int grp = blockIdx.x / segs, seg = blockIdx.x - grp * segs;
  return {static_cast<int64_t>(grp) * (kThreads >> lg) + (threadIdx.x >> lg),
          ((seg << lg) + static_cast<int>(threadIdx.x & ((1 << lg) - 1))) * kV};
}
// Rows that hold work: all P, or what the caller's device counter says.
__device__ __forceinline__ int64_t rows_used(int P, const int32_t* n_rows) {
  return n_rows ? min(P, max(*n_rows, 0)) : P;
}

// silu(z) = z / (1 + e^-z) with its logistic factor.
__device__ __forceinline__ float logistic(float z) { return 1.0f / (1.0f + expf(-z)); }

enum SwigluOut { kSame, kCodesOut };

template <bool F32, int OUT>
__global__ __launch_bounds__(kThreads) void swiglu_rows(int P, int f, int segs, int lg,
                                                        const void* gu, void* h, float* scales,
                                                        const int32_t* n_rows) {
  const Spot s = spot(segs, lg);
  const bool in = s.row < rows_used(P, n_rows) && s.c < f;
  float o[kV] = {};
  if (in) {
    float g[kV], u[kV];
    load8<F32>(gu, s.row * 2 * f + s.c, g);
    load8<F32>(gu, s.row * 2 * f + f + s.c, u);
#pragma unroll
    for (int j = 0; j < kV; ++j) o[j] = silu(g[j]) * u[j];
  }
  if constexpr (OUT == kSame) {
    if (in) store8<F32>(h, s.row * f + s.c, o);
  } else {
    const int n = scale_exponent(group_max(absmax8(o)));
    if (in) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(h) + s.row * f + s.c) = codes8(o, n);
      if (threadIdx.x % kGroupLanes == 0)
        scales[s.row * ((f + kBlock - 1) / kBlock) + s.c / kBlock] = two_to(n);
    }
  }
}

// dg = dh u s (1 + g (1 - s)), du = dh g s with s = 1 / (1 + e^-g).
template <bool F32>
__global__ __launch_bounds__(kThreads) void swiglu_grad_rows(int P, int f, int segs, int lg,
                                                             const void* gu, const void* dh,
                                                             void* dgu, const int32_t* n_rows) {
  const Spot s = spot(segs, lg);
  if (s.row >= rows_used(P, n_rows) || s.c >= f) return;
  float g[kV], u[kV], d[kV], dg[kV], du[kV];
  load8<F32>(gu, s.row * 2 * f + s.c, g);
  load8<F32>(gu, s.row * 2 * f + f + s.c, u);
  load8<F32>(dh, s.row * f + s.c, d);
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    const float sg = logistic(g[j]);
    dg[j] = d[j] * u[j] * (sg * fmaf(g[j], 1.0f - sg, 1.0f));
    du[j] = d[j] * (g[j] * sg);
  }
  store8<F32>(dgu, s.row * 2 * f + s.c, dg);
  store8<F32>(dgu, s.row * 2 * f + f + s.c, du);
}

struct RowGrid {
  int segs, lg;
  dim3 grid;
};
RowGrid row_grid(int P, int f) {
  RowGrid r;
  r.lg = 4;  // at least the 16 lanes of a scale block
  while ((1 << r.lg) < kThreads && (1 << r.lg) * kV < f) ++r.lg;
  r.segs = (f / kV + (1 << r.lg) - 1) >> r.lg;
  const int per = kThreads >> r.lg;
  r.grid = dim3(static_cast<uint32_t>((P + per - 1) / per) * r.segs);
  return r;
}

}  // namespace

hipError_t launch_blockscale_quantize(int n_mats, int R, int K, const void* x, bool f32,
                                      bool square, uint8_t* codes, float* scales,
                                      hipStream_t stream) {
  const int KB = (K + kBlock - 1) / kBlock;
  const dim3 block(kThreads);
  if (square) {
    const int RB = (R + kBlock - 1) / kBlock;
    const dim3 grid(static_cast<uint32_t>(static_cast<int64_t>(n_mats) * RB * KB));
    return f32 ? launch(quant_blocks<true>, grid, block, 0, stream, R, K, RB, KB, x, codes, scales)
               : launch(quant_blocks<false>, grid, block, 0, stream, R, K, RB, KB, x, codes,
                        scales);
  }
  const int64_t blocks = static_cast<int64_t>(n_mats) * R * KB;
  const int per = kThreads / kGroupLanes;
  const dim3 grid(static_cast<uint32_t>((blocks + per - 1) / per));
  return f32 ? launch(quant_rows<true>, grid, block, 0, stream, blocks, K, KB, x, codes, scales)
             : launch(quant_rows<false>, grid, block, 0, stream, blocks, K, KB, x, codes, scales);
}

hipError_t launch_swiglu(int P, int f, const void* gu, bool f32, void* h, float* scales,
                         const int32_t* n_rows, hipStream_t stream) {
  const RowGrid r = row_grid(P, f);
  const dim3 block(kThreads);
  if (scales)
    return f32 ? launch(swiglu_rows<true, kCodesOut>, r.grid, block, 0, stream, P, f, r.segs, r.lg,
                        gu, h, scales, n_rows)
               : launch(swiglu_rows<false, kCodesOut>, r.grid, block, 0, stream, P, f, r.segs,
                        r.lg, gu, h, scales, n_rows);
  return f32 ? launch(swiglu_rows<true, kSame>, r.grid, block, 0, stream, P, f, r.segs, r.lg, gu,
                      h, scales, n_rows)
             : launch(swiglu_rows<false, kSame>, r.grid, block, 0, stream, P, f, r.segs, r.lg, gu,
                      h, scales, n_rows);
}

hipError_t launch_swiglu_grad(int P, int f, const void* gu, const void* dh, bool f32, void* dgu,
                              const int32_t* n_rows, hipStream_t stream) {
  const RowGrid r = row_grid(P, f);
  const dim3 block(kThreads);
  return f32 ? launch(swiglu_grad_rows<true>, r.grid, block, 0, stream, P, f, r.segs, r.lg, gu, dh,
                      dgu, n_rows)
             : launch(swiglu_grad_rows<false>, r.grid, block, 0, stream, P, f, r.segs, r.lg, gu,
                      dh, dgu, n_rows);
}

}  // namespace moe
