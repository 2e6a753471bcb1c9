// One AdamW step over many tensors, its moments in float32 or in 8 bits.
//
//   g' = grad_scale * g
//   m  = b1 m + (1 - b1) g'            v = b2 v + (1 - b2) g'^2
//   p  = p (1 - lr * decay) - size * m / (sqrt(v) * root + eps)
//   size = lr / (1 - b1^t), root = 1 / sqrt(1 - b2^t)
//
// in float32, each operation rounded (b1^t and b2^t in double), so that the
// result does not depend on how a tensor is cut into work.
//
// 8 bits: 256 elements share a power of two for each moment.  m is e4m3 codes
// (the scale the smallest that keeps the block within 448).  Of v its root is
// held, whose range is half of v's in the exponent: code c = 32 e + t stands for
// t 2^e, e 0..6 and t up to 63 (from 32 on where e > 0): 6 significant bits over a
// range of 2^12, the scale the smallest that keeps the block within 4032.  A root
// that is not zero never gets code 0: m, whose codes reach further down, would
// then be divided by eps alone.
//
// Bound by memory: a wavefront takes blocks of 256 elements, 4 of each lane, and
// reads several of them before it works on the first.  The tensors' addresses
// are kernel arguments (a batch of them a launch): nothing is kept on the device,
// and a captured launch holds them.
#include "common.h"
#include "launch.h"

#pragma clang fp contract(off)  // every product and sum is rounded, as the formulas say

namespace moe {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr int kV = 4;                // elements per lane of a block
constexpr int kBlock = kWave * kV;   // elements per scale
static_assert(kBlock == kAdamWBlock, "a wavefront holds a block");
constexpr uint32_t kMaxGrid = 1u << 22;

enum Store { kF32, kBf16, kMaster };  // the parameter: float32, bf16, bf16 with a float32 master

struct Batch {
  AdamWTensor t[kAdamWBatch];
  uint32_t first[kAdamWBatch + 1];  // each tensor's first chunk; the last: how many there are
  int n;
  AdamWStep s;
};

__device__ __forceinline__ float two_to(int n) {
  return __uint_as_float(static_cast<uint32_t>(n + 127) << 23);
}
__device__ __forceinline__ bool finite(float v) {
  return (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u;
}

// Elements i .. i + 3 of an array of n; `wide`: it is aligned for one access.
template <class T>
__device__ __forceinline__ void load4(const T* p, int64_t i, int64_t n, bool wide, T (&v)[kV]) {
  struct alignas(sizeof(T) * kV) Pack {
    T v[kV];
  };
  if (wide && i + kV <= n) {
    const Pack q = *reinterpret_cast<const Pack*>(p + i);
#pragma unroll
    for (int j = 0; j < kV; ++j) v[j] = q.v[j];
  } else {
#pragma unroll
    for (int j = 0; j < kV; ++j) v[j] = i + j < n ? p[i + j] : T(0);
  }
}
template <class T>
__device__ __forceinline__ void store4(T* p, int64_t i, int64_t n, bool wide, const T (&v)[kV]) {
  struct alignas(sizeof(T) * kV) Pack {
    T v[kV];
  };
  if (wide && i + kV <= n) {
    Pack q;
#pragma unroll
    for (int j = 0; j < kV; ++j) q.v[j] = v[j];
    *reinterpret_cast<Pack*>(p + i) = q;
  } else {
#pragma unroll
    for (int j = 0; j < kV; ++j)
      if (i + j < n) p[i + j] = v[j];
  }
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  for (int off = kWave / 2; off > 0; off >>= 1)
    v = max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), off, kWave)));
  return v;
}

// Exponent n of the smallest scale 2^n >= 2^-126 with top <= limit * 2^n, limit =
// 1.mant * 2^log: 0 for a top of zero.
__device__ __forceinline__ int scale_exponent(uint32_t top, uint32_t mant, int log) {
  if (top == 0u) return 0;
  const int e = static_cast<int>(top >> 23) - 127;
  return max(-126, (top & 0x7FFFFFu) <= mant ? e - log : e - log + 1);
}

// What a lane holds of a block before its update.
template <bool B8, int P, bool GBF16>
struct Loaded {
  float p32[kV];
  uint16_t p16[kV], g16[kV];
  float g32[kV], m32[kV], v32[kV];
  uint8_t mc[kV], vc[kV];
  float ms, vs;
};

template <bool B8, int P, bool GBF16, int U>
__global__ __launch_bounds__(kThreads) void adamw_step(const Batch b) {
  const int lane = threadIdx.x & (kWave - 1);
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t my_first = b.first[min(lane, b.n)];
  const uint32_t chunks = b.first[b.n];
  const double t = static_cast<double>(max(*b.s.step, int64_t(1)));
  const float size = static_cast<float>(b.s.lr / (1.0 - exp(t * b.s.log_beta1)));
  const float root = static_cast<float>(1.0 / sqrt(1.0 - exp(t * b.s.log_beta2)));
  const float gs = b.s.grad_scale ? *b.s.grad_scale : 1.0f;
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    // the last tensor whose first chunk is not behind c
    const int at = __popcll(__ballot(lane < b.n && my_first <= c)) - 1;
    const AdamWTensor q = b.t[at];
    const int64_t n = q.n;
    const bool wide = q.wide;
    const int64_t from =
        (static_cast<int64_t>(c - b.first[at]) * (kWaves * U) + wv * U) * kBlock + lane * kV;
    Loaded<B8, P, GBF16> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = from + u * kBlock;
      if (P == kF32) load4(static_cast<const float*>(q.p), i, n, wide, x[u].p32);
      if (P == kBf16) load4(static_cast<const uint16_t*>(q.p), i, n, wide, x[u].p16);
      if (P == kMaster) load4(static_cast<const float*>(q.master), i, n, wide, x[u].p32);
      if (GBF16)
        load4(static_cast<const uint16_t*>(q.g), i, n, wide, x[u].g16);
      else
        load4(static_cast<const float*>(q.g), i, n, wide, x[u].g32);
      if (B8) {
        load4(static_cast<const uint8_t*>(q.m), i, n, wide, x[u].mc);
        load4(static_cast<const uint8_t*>(q.v), i, n, wide, x[u].vc);
        const int64_t blk = (from - lane * kV) / kBlock + u;
        const bool in = blk * kBlock < n;
        x[u].ms = in ? q.m_scales[blk] : 0.0f;
        x[u].vs = in ? q.v_scales[blk] : 0.0f;
      } else {
        load4(static_cast<const float*>(q.m), i, n, wide, x[u].m32);
        load4(static_cast<const float*>(q.v), i, n, wide, x[u].v32);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = from + u * kBlock;
      float m[kV], v[kV], r[kV], p[kV];
      if (B8) {
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < kV; ++j) w |= static_cast<uint32_t>(x[u].mc[j]) << (8 * j);
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
        const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
        m[0] = lo[0] * x[u].ms; m[1] = lo[1] * x[u].ms;
        m[2] = hi[0] * x[u].ms; m[3] = hi[1] * x[u].ms;
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          const int code = x[u].vc[j], e = max((code >> 5) - 1, 0);
          const float s = static_cast<float>((code - 32 * e) << e) * x[u].vs;
          v[j] = s * s;
        }
      } else {
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          m[j] = x[u].m32[j];
          v[j] = x[u].v32[j];
        }
      }
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        float g = GBF16 ? bf16_to_f32(x[u].g16[j]) : x[u].g32[j];
        g = g * gs;
        m[j] = m[j] * b.s.beta1 + g * b.s.rest1;
        v[j] = v[j] * b.s.beta2 + g * g * b.s.rest2;
        r[j] = sqrtf(v[j]);
        p[j] = P == kBf16 ? bf16_to_f32(x[u].p16[j]) : x[u].p32[j];
        p[j] = p[j] * b.s.keep - m[j] / (r[j] * root + b.s.eps) * size;
      }
      if (P != kF32) {
        uint16_t h[kV];
#pragma unroll
        for (int j = 0; j < kV; ++j) h[j] = f32_to_bf16(p[j]);
        store4(static_cast<uint16_t*>(q.p), i, n, wide, h);
      }
      if (P != kBf16) store4(static_cast<float*>(P == kMaster ? q.master : q.p), i, n, wide, p);
      if (B8) {
        uint32_t top_m = 0, top_r = 0;
#pragma unroll
        for (int j = 0; j < kV; ++j)
          if (i + j < n) {
            if (finite(m[j])) top_m = max(top_m, __float_as_uint(m[j]) & 0x7FFFFFFFu);
            top_r = max(top_r, __float_as_uint(r[j]) & 0x7FFFFFFFu);
          }
        top_m = wave_max(top_m);
        top_r = wave_max(top_r);
        const int em = scale_exponent(top_m, 0x600000u, 8);   // 448 = 1.75 * 2^8
        const int er = scale_exponent(top_r, 0x7C0000u, 11);  // 4032 = 1.96875 * 2^11
        const bool ok = top_r < 0x7F800000u;
        const float im = two_to(-em), ir = ok ? two_to(-er) : 0.0f;
        uint8_t mc[kV], vc[kV];
        float a[kV];
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          a[j] = finite(m[j]) ? m[j] * im : __uint_as_float(0x7FC00000u);
          const float s = ok ? r[j] * ir : 0.0f;
          const int e = max(static_cast<int>(__float_as_uint(s) >> 23) - 126 - 6, 0);
          const int code = 32 * e + static_cast<int>(rintf(s * two_to(-e)));
          vc[j] = static_cast<uint8_t>(r[j] > 0.0f ? max(code, 1) : code);
        }
        int w = 0;
        w = __builtin_amdgcn_cvt_pk_fp8_f32(a[0], a[1], w, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(a[2], a[3], w, true);
#pragma unroll
        for (int j = 0; j < kV; ++j) mc[j] = static_cast<uint8_t>(w >> (8 * j));
        store4(static_cast<uint8_t*>(q.m), i, n, wide, mc);
        store4(static_cast<uint8_t*>(q.v), i, n, wide, vc);
        const int64_t blk = (from - lane * kV) / kBlock + u;
        if (lane == 0 && blk * kBlock < n) {
          q.m_scales[blk] = two_to(em);
          q.v_scales[blk] = ok ? two_to(er) : __uint_as_float(0x7FC00000u);
        }
      } else {
        store4(static_cast<float*>(q.m), i, n, wide, m);
        store4(static_cast<float*>(q.v), i, n, wide, v);
      }
    }
  }
}

// Four blocks a wavefront, one where they would not fill the CUs twice.
constexpr int64_t kFewElements = 2 * 256 * kWaves * 4 * kBlock;

template <bool B8, int P, bool GBF16>
hipError_t go(const Batch& b, bool few, hipStream_t stream) {
  const uint32_t chunks = b.first[b.n];
  const dim3 grid(chunks < kMaxGrid ? chunks : kMaxGrid), block(kThreads);
  return few ? launch(adamw_step<B8, P, GBF16, 1>, grid, block, 0, stream, b)
             : launch(adamw_step<B8, P, GBF16, 4>, grid, block, 0, stream, b);
}

template <bool B8>
hipError_t go(const Batch& b, int store, bool gbf16, bool few, hipStream_t stream) {
  switch (store) {
    case kF32: return gbf16 ? go<B8, kF32, true>(b, few, stream) : go<B8, kF32, false>(b, few, stream);
    case kBf16:
      return gbf16 ? go<B8, kBf16, true>(b, few, stream) : go<B8, kBf16, false>(b, few, stream);
    default:
      return gbf16 ? go<B8, kMaster, true>(b, few, stream) : go<B8, kMaster, false>(b, few, stream);
  }
}

}  // namespace

// Tensors of one kind (how the parameter, its gradient and its moments are held)
// share launches, up to kAdamWBatch at a time.
hipError_t launch_adamw(const AdamWSource& src, int n, const AdamWStep& s, hipStream_t stream) {
  int64_t total = 0;
  for (int i = 0; i < n; ++i) total += src.get(src.tensors, i).n;
  const bool few = total < kFewElements;
  const int64_t per = static_cast<int64_t>(kWaves) * (few ? 1 : 4) * kBlock;
  for (int kind = 0; kind < 12; ++kind) {
    Batch b;
    b.n = 0;
    b.first[0] = 0;
    b.s = s;
    auto flush = [&]() -> hipError_t {
      if (b.n == 0) return hipSuccess;
      const int store = kind >> 2;
      const bool b8 = kind & 1, gbf16 = kind & 2;
      const hipError_t e = b8 ? go<true>(b, store, gbf16, few, stream)
                              : go<false>(b, store, gbf16, few, stream);
      b.n = 0;
      return e;
    };
    for (int i = 0; i < n; ++i) {
      const AdamWTensor t = src.get(src.tensors, i);
      const int store = t.master ? kMaster : t.p_bf16 ? kBf16 : kF32;
      if (t.n == 0 || (store << 2 | t.g_bf16 << 1 | (t.m_scales != nullptr)) != kind) continue;
      const int64_t chunks = (t.n + per - 1) / per;
      if (b.n == kAdamWBatch || (b.n > 0 && b.first[b.n] + chunks > INT32_MAX)) {
        const hipError_t e = flush();
        if (e != hipSuccess) return e;
      }
      b.t[b.n] = t;
      b.first[b.n + 1] = b.first[b.n] + static_cast<uint32_t>(chunks);
      ++b.n;
    }
    const hipError_t e = flush();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
