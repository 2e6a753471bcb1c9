// 8-bit floats with a scale per block of 128: rows (1 x 128, activations) or
// 128 x 128 (weights) to e4m3 codes and float32 scales, and SwiGLU over
// grouped rows (also straight to codes) with its gradient.
//
// The scale is a power of two, the smallest that keeps the block's largest
// magnitude within 448 (e4m3's largest): dividing by it is exact, so every
// code is the value rounded once, and no rounding of a quotient can move it.
// e4m3 is a floating format, so a scale that is not exactly absmax / 448 costs
// no precision outside its subnormals.
//
// Bound by memory: a thread takes 8 columns, 16 lanes a block.  SwiGLU of the
// 2048-token prompt (16,384 rows of 2 x 2048 bf16, 201 MB) takes 34 us (5.9
// TB/s, part of it from the caches), its gradient over 32,744 rows of 2 x 1024
// (335 MB) 58 us (5.7 TB/s); straight to codes the prompt's SwiGLU (169 MB) takes
// 43 us.  2048 rows of 6144 are quantised in 10 us, 64 matrices of 2048 x 2048 by
// 128 x 128 (0.81 GB) in 173 (4.6 TB/s).
#include "common.h"
#include "launch.h"

#pragma clang fp contract(off)  // the fused multiply-adds are written out

namespace moe {

namespace {

constexpr int kV = 8;         // columns per thread
constexpr int kBlock = 128;   // columns per scale
constexpr int kGroupLanes = kBlock / kV;
constexpr int kThreads = 256;
// Workgroups of a launch at most (a grid holds fewer than 2^32 threads); each
// takes several places where there are more.
constexpr int64_t kMaxGrid = int64_t(1) << 22;

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
  constexpr int kPer = kThreads / kGroupLanes;
  for (int64_t b = static_cast<int64_t>(blockIdx.x) * kPer + threadIdx.x / kGroupLanes; b < blocks;
       b += static_cast<int64_t>(gridDim.x) * kPer) {
    const int64_t row = b / KB;
    const int c = static_cast<int>(b - row * KB) * kBlock + (threadIdx.x % kGroupLanes) * kV;
    float v[kV] = {};
    if (c < K) load8<F32>(x, row * K + c, v);
    const int n = scale_exponent(group_max(absmax8(v)));
    if (c < K) *reinterpret_cast<uint2*>(codes + row * K + c) = codes8(v, n);
    if (threadIdx.x % kGroupLanes == 0) scales[b] = two_to(n);
  }
}

// 128 x 128: one workgroup per block, 8 rows of 8 columns per thread.
template <bool F32>
__global__ __launch_bounds__(kThreads) void quant_blocks(int64_t blocks, int R, int K, int RB,
                                                         int KB, const void* __restrict__ x,
                                                         uint8_t* __restrict__ codes,
                                                         float* __restrict__ scales) {
  __shared__ float sh[kThreads / kWave];
  constexpr int kRows = kThreads / kGroupLanes;  // rows per pass
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
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
    __syncthreads();
    const int n = scale_exponent(m);
#pragma unroll
    for (int i = 0; i < kBlock / kRows; ++i)
      if (c < K && r0 + i * kRows < R)
        *reinterpret_cast<uint2*>(codes + (base + r0 + i * kRows) * K + c) = codes8(v[i], n);
    if (threadIdx.x == 0) scales[b] = two_to(n);
  }
}

// A launch over rows: `segs` workgroups per group of rows, 2^lg threads per
// row, the groups of rows in turns of the grid.  f(row, first column) by every
// thread of the workgroup together, also past the last row or column.
struct RowGrid {
  int segs, lg;
  int step;  // groups of rows per turn of the grid; 0: one turn takes all
};
template <class F>
__device__ __forceinline__ void for_rows(const RowGrid& r, int64_t rows, F f) {
  const int per = kThreads >> r.lg, grp = blockIdx.x / r.segs, seg = blockIdx.x - grp * r.segs;
  const int c = ((seg << r.lg) + static_cast<int>(threadIdx.x & ((1 << r.lg) - 1))) * kV;
  int64_t first = static_cast<int64_t>(grp) * per;
  f(first + (threadIdx.x >> r.lg), c);
  if (r.step == 0) return;  // one turn (as a loop of one, the gradient took 64 us instead of 60)
  for (first += static_cast<int64_t>(r.step) * per; first < rows;
       first += static_cast<int64_t>(r.step) * per)
    f(first + (threadIdx.x >> r.lg), c);
}
// Rows that hold work: all P, or what the caller's device counter says.
__device__ __forceinline__ int64_t rows_used(int P, const int32_t* n_rows) {
  return n_rows ? min(P, max(*n_rows, 0)) : P;
}

// silu(z) = z / (1 + e^-z) with its logistic factor.
__device__ __forceinline__ float logistic(float z) { return 1.0f / (1.0f + expf(-z)); }

enum SwigluOut { kSame, kCodesOut };

template <bool F32, int OUT>
__global__ __launch_bounds__(kThreads) void swiglu_rows(int P, int f, RowGrid rg, const void* gu,
                                                        void* h, float* scales,
                                                        const int32_t* n_rows) {
  const int64_t rows = rows_used(P, n_rows);
  for_rows(rg, rows, [&](int64_t row, int c) {
    const bool in = row < rows && c < f;
    float o[kV] = {};
    if (in) {
      float g[kV], u[kV];
      load8<F32>(gu, row * 2 * f + c, g);
      load8<F32>(gu, row * 2 * f + f + c, u);
#pragma unroll
      for (int j = 0; j < kV; ++j) o[j] = silu(g[j]) * u[j];
    }
    if constexpr (OUT == kSame) {
      if (in) store8<F32>(h, row * f + c, o);
    } else {
      const int n = scale_exponent(group_max(absmax8(o)));
      if (in) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(h) + row * f + c) = codes8(o, n);
        if (threadIdx.x % kGroupLanes == 0)
          scales[row * ((f + kBlock - 1) / kBlock) + c / kBlock] = two_to(n);
      }
    }
  });
}

// dg = dh u s (1 + g (1 - s)), du = dh g s with s = 1 / (1 + e^-g).
template <bool F32>
__global__ __launch_bounds__(kThreads) void swiglu_grad_rows(int P, int f, RowGrid rg,
                                                             const void* gu, const void* dh,
                                                             void* dgu, const int32_t* n_rows) {
  const int64_t rows = rows_used(P, n_rows);
  for_rows(rg, rows, [&](int64_t row, int c) {
    if (row >= rows || c >= f) return;
    float g[kV], u[kV], d[kV], dg[kV], du[kV];
    load8<F32>(gu, row * 2 * f + c, g);
    load8<F32>(gu, row * 2 * f + f + c, u);
    load8<F32>(dh, row * f + c, d);
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const float sg = logistic(g[j]);
      dg[j] = d[j] * u[j] * (sg * fmaf(g[j], 1.0f - sg, 1.0f));
      du[j] = d[j] * (g[j] * sg);
    }
    store8<F32>(dgu, row * 2 * f + c, dg);
    store8<F32>(dgu, row * 2 * f + f + c, du);
  });
}

struct RowLaunch {
  RowGrid rg;
  dim3 grid;
};
RowLaunch row_launch(int P, int f) {
  RowLaunch r;
  r.rg.lg = 4;  // at least the 16 lanes of a scale block
  while ((1 << r.rg.lg) < kThreads && (1 << r.rg.lg) * kV < f) ++r.rg.lg;
  r.rg.segs = (f / kV + (1 << r.rg.lg) - 1) >> r.rg.lg;
  const int per = kThreads >> r.rg.lg;
  const int64_t groups = (P + per - 1) / per, most = kMaxGrid / r.rg.segs;
  r.rg.step = groups <= most ? 0 : static_cast<int>(most);
  r.grid = dim3(static_cast<uint32_t>(groups <= most ? groups : most) * r.rg.segs);
  return r;
}

}  // namespace

hipError_t launch_blockscale_quantize(int n_mats, int R, int K, const void* x, bool f32,
                                      bool square, uint8_t* codes, float* scales,
                                      hipStream_t stream) {
  const int KB = (K + kBlock - 1) / kBlock, RB = (R + kBlock - 1) / kBlock;
  const dim3 block(kThreads);
  const int64_t blocks = static_cast<int64_t>(n_mats) * (square ? RB : R) * KB;
  const int per = square ? 1 : kThreads / kGroupLanes;
  const int64_t groups = (blocks + per - 1) / per;
  const dim3 grid(static_cast<uint32_t>(groups < kMaxGrid ? groups : kMaxGrid));
  if (square)
    return launch(f32 ? quant_blocks<true> : quant_blocks<false>, grid, block, 0, stream, blocks, R,
                  K, RB, KB, x, codes, scales);
  return launch(f32 ? quant_rows<true> : quant_rows<false>, grid, block, 0, stream, blocks, K, KB,
                x, codes, scales);
}

hipError_t launch_swiglu(int P, int f, const void* gu, bool f32, void* h, float* scales,
                         const int32_t* n_rows, hipStream_t stream) {
  const RowLaunch r = row_launch(P, f);
  auto go = [&](auto kernel) {
    return launch(kernel, r.grid, dim3(kThreads), 0, stream, P, f, r.rg, gu, h, scales, n_rows);
  };
  if (scales) return f32 ? go(swiglu_rows<true, kCodesOut>) : go(swiglu_rows<false, kCodesOut>);
  return f32 ? go(swiglu_rows<true, kSame>) : go(swiglu_rows<false, kSame>);
}

hipError_t launch_swiglu_grad(int P, int f, const void* gu, const void* dh, bool f32, void* dgu,
                              const int32_t* n_rows, hipStream_t stream) {
  const RowLaunch r = row_launch(P, f);
  return launch(f32 ? swiglu_grad_rows<true> : swiglu_grad_rows<false>, r.grid, dim3(kThreads), 0,
                stream, P, f, r.rg, gu, dh, dgu, n_rows);
}

}  // namespace moe
