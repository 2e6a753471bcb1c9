// 8-bit integers with a float32 scale per row: float rows (tokens, or a weight
// matrix's output channels) to codes, and SwiGLU over grouped rows straight to
// them.
//
//   scale = max(absmax * (1 / 127), 2^-126)     (1 for a row of zeros)
//   code  = the integer nearest to x / scale, ties to even
//
// The quotient is not formed: q = rint(x * (1 / scale)) is within one of the
// code, and r = x - q * scale, one fused multiply-add, is exact (r is a multiple
// of the smaller of x's and scale's last places and hardly larger than half of
// scale), so comparing r with scale / 2 decides the code exactly.
// A row that holds an infinity or a NaN has no scale: it becomes NaN, which
// every product with the row's codes (zeros) then is.
//
// Bound by memory.  A row is read once and stays in registers between its
// largest magnitude and its codes: a wavefront's where it has at most 2048
// columns, a workgroup's up to 8192, and wider ones are read again.  Measured:
// 16,384 rows of SwiGLU to 2048 codes 38 us (168 MB, 4.4 TB/s; 45 with every code
// compared), 2048 rows of 6144 10 us (38 MB, mostly the launch and one row's way).
#include "common.h"
#include "launch.h"

#pragma clang fp contract(off)  // the fused multiply-adds are written out

namespace moe {

namespace {

constexpr int kV = 8;  // columns per thread and chunk
constexpr int kThreads = 256;
constexpr int kHeld = 4;  // chunks a thread keeps
constexpr int64_t kMaxGrid = int64_t(1) << 22;  // a grid holds fewer than 2^32 threads

template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[kV]) {
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

// Eight columns of a row, as the codes' source.
template <bool F32, bool SWIGLU>
struct Row {
  const void* p;
  int64_t at;  // the row's first value (of gate)
  int K;
  __device__ __forceinline__ void load(int c, float (&v)[kV]) const {
    load8<F32>(p, at + c, v);
    if constexpr (SWIGLU) {
      float u[kV];
      load8<F32>(p, at + K + c, u);
#pragma unroll
      for (int j = 0; j < kV; ++j) v[j] = silu(v[j]) * u[j];
    }
  }
};

// The largest magnitude's bits; at least infinity's where one is not finite.
__device__ __forceinline__ uint32_t top8(const float (&v)[kV], uint32_t m) {
#pragma unroll
  for (int j = 0; j < kV; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  return m;
}

constexpr uint32_t kInfinity = 0x7F800000u;

__device__ __forceinline__ float row_scale(uint32_t top) {
  if (top == 0u) return 1.0f;
  if (top >= kInfinity) return __uint_as_float(0x7FC00000u);
  return fmaxf(__uint_as_float(top) * (1.0f / 127.0f), 0x1p-126f);
}

// Eight codes; zeros where the scale is NaN.  Quotients this near to a half-way
// point (about one wavefront's codes in twenty hold one) are decided by r.
__device__ __forceinline__ uint2 codes8(const float (&v)[kV], float scale) {
  if (!(scale == scale)) return make_uint2(0u, 0u);
  const float inv = 1.0f / scale, half = 0.5f * scale, near = 0.9999f * half;
  float q[kV];
  bool close = false;
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    q[j] = rintf(v[j] * inv);
    close = close || fabsf(fmaf(-q[j], scale, v[j])) > near;
  }
  if (close) {
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const float r = fmaf(-q[j], scale, v[j]);
      const bool odd = static_cast<int>(q[j]) & 1;
      if (r > half || (r == half && odd)) q[j] += 1.0f;
      if (r < -half || (r == -half && odd)) q[j] -= 1.0f;
    }
  }
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < kV; ++j)
    w[j / 4] |= (static_cast<uint32_t>(static_cast<int>(q[j])) & 0xFFu) << (8 * (j % 4));
  return make_uint2(w[0], w[1]);
}

// WIDE: a workgroup per row, else a wavefront.
template <bool F32, bool SWIGLU, bool WIDE>
__global__ __launch_bounds__(kThreads) void row_codes(int64_t rows, int K,
                                                      const void* __restrict__ x,
                                                      uint8_t* __restrict__ codes,
                                                      float* __restrict__ scales,
                                                      const int32_t* __restrict__ n_rows) {
  constexpr int kTeam = WIDE ? kThreads : kWave, kPer = kThreads / kTeam;
  __shared__ uint32_t sh[2][kThreads / kWave];
  const int t = threadIdx.x % kTeam;
  const int64_t used = n_rows ? min(rows, static_cast<int64_t>(max(*n_rows, 0))) : rows;
  int turn = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kPer + threadIdx.x / kTeam; row < used;
       row += static_cast<int64_t>(gridDim.x) * kPer, turn ^= 1) {
    const Row<F32, SWIGLU> src{x, row * K * (SWIGLU ? 2 : 1), K};
    float v[kHeld][kV];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int c = (i * kTeam + t) * kV;
      if (c < K) {
        src.load(c, v[i]);
        m = top8(v[i], m);
      }
    }
    for (int c = (kHeld * kTeam + t) * kV; c < K; c += kTeam * kV) {
      float u[kV];
      src.load(c, u);
      m = top8(u, m);
    }
    m = wave_max_u32(m);
    if constexpr (WIDE) {  // two turns' maxima in turn, so one meeting each is enough
      if (threadIdx.x % kWave == 0) sh[turn][threadIdx.x / kWave] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kThreads / kWave; ++w) m = max(m, sh[turn][w]);
    }
    const float scale = row_scale(m);
    uint8_t* out = codes + row * K;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int c = (i * kTeam + t) * kV;
      if (c < K) *reinterpret_cast<uint2*>(out + c) = codes8(v[i], scale);
    }
    for (int c = (kHeld * kTeam + t) * kV; c < K; c += kTeam * kV) {
      float u[kV];
      src.load(c, u);
      *reinterpret_cast<uint2*>(out + c) = codes8(u, scale);
    }
    if (t == 0) scales[row] = scale;
  }
}

template <bool SWIGLU>
hipError_t go(int64_t rows, int K, const void* x, bool f32, uint8_t* codes, float* scales,
              const int32_t* n_rows, hipStream_t stream) {
  const bool wide = K > kHeld * kWave * kV;
  const int64_t per = wide ? 1 : kThreads / kWave, groups = (rows + per - 1) / per;
  const dim3 grid(static_cast<uint32_t>(groups < kMaxGrid ? groups : kMaxGrid));
  auto run = [&](auto kernel) {
    return launch(kernel, grid, dim3(kThreads), 0, stream, rows, K, x, codes, scales, n_rows);
  };
  if (f32) return wide ? run(row_codes<true, SWIGLU, true>) : run(row_codes<true, SWIGLU, false>);
  return wide ? run(row_codes<false, SWIGLU, true>) : run(row_codes<false, SWIGLU, false>);
}

}  // namespace

hipError_t launch_rowscale_quantize(int64_t rows, int K, const void* x, bool f32, uint8_t* codes,
                                    float* scales, hipStream_t stream) {
  return go<false>(rows, K, x, f32, codes, scales, nullptr, stream);
}

hipError_t launch_swiglu_rowscale(int P, int f, const void* gu, bool f32, uint8_t* codes,
                                  float* scales, const int32_t* n_rows, hipStream_t stream) {
  return go<true>(P, f, gu, f32, codes, scales, n_rows, stream);
}

}  // namespace moe
