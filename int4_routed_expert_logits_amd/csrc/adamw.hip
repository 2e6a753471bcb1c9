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
// then be divided by eps alone.  Where an element's root is not finite, its block's
// scale is a NaN that carries the scale's exponent in its last 8 bits, and code
// 255 stands for infinity (the other codes keep below it): that element stays so
// (its m has no part in m's scale), the 255 beside it are as they would be without it.
//
// How codes are rounded.  A step moves v by (1 - b2)(g'^2 - v) at most and m by
// (1 - b1)(g' - m); rounded to nearest, a code stays where it is if that is less
// than half a place, in the next step too, and a moment that should fall or grow
// slowly never does.  So the codes are rounded up or down with the probability that
// makes the expected m and the expected v (not its root) the ones rounded, the draw
// a hash of the step's number and the element's place: the same state gives the same
// bits, and over steps the errors cancel.  A root's own spread from it is 6 to 8%
// down to a thirtieth of its block's largest, 10% at a hundredth, 32% at a
// thousandth.  Norm of the update over the one with float32 moments after 3000 steps
// (nearest / by the hash, b1 = 0.9; normal gradients, constant ones of mixed sizes,
// and normal ones 20 times smaller after a third):
//   b2 = 0.95   1.01 / 1.00   0.88 / 1.00   1.01 / 1.00
//   b2 = 0.99   0.61 / 1.01   1.34 / 1.00   0.03 / 1.01
//   b2 = 0.999  1.49 / 1.01   3.39 / 1.00   0.69 / 1.05
// Codes go to the nearest, which needs fewer instructions (1375 against 1530 us for
// 402M elements with masters), where that keeps the norm within 12%: with b2 <= 0.95,
// so that v falls, and 1 - b2 between a half and a fifth of 1 - b1, where the two
// moments' lags behind constant gradients nearly cancel (b1 / b2 of 0.9 / 0.95: 0.88
// to 0.98, 0.8 / 0.9: 0.90 to 0.99, 0.7 / 0.94: 1.04 to 1.09, 0.5 / 0.9: 1.06 to 1.09;
// but 0.9 / 0.9: 0.79 to 0.88, 0.5 / 0.95: 1.13 to 1.21).
//
// Bound by memory: 402M elements of bf16 with masters take 2.25 ms (30 bytes each,
// 5.4 TB/s), with 8-bit moments 1.37 (18 bytes, 5.3 TB/s; 473 vector instructions a
// wavefront fill the SIMDs beside it), hashed 1.53 (601, which bound it); few
// elements by the launch and by the betas' powers, which each wavefront computes in
// double ahead of its data (16 vectors of 6144: 3.6 us).  A wavefront takes one block
// of 256 elements, 4 of each lane: with so many wavefronts in flight, four blocks
// each before the first is worked on gain nothing (2.26 and 1.41 ms), and starve
// where there are few (90 odd tensors, 2.9M elements: 28 us on the GPU, so 17).  The
// tensors' addresses are kernel arguments, up to 64 tensors a launch: nothing is
// kept on the device, and a captured launch holds them.
#include <utility>

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
enum Moments { kFloats, kNearest, kHashed };  // float32; codes, and how they are rounded

// The tensors of a launch, by what their kind has of addresses: as many as the
// 4 KB of a launch's arguments hold, and a wavefront's lanes.
template <bool B8, int P>
struct Batch {
  static constexpr int kPtrs = 4 + (P == kMaster) + 2 * B8;
  static constexpr int kFit = (4096 - 128) / (8 * (kPtrs + 1) + 4);
  static constexpr int kMost = kFit < kWave ? kFit : kWave;
  struct Slot {
    uint64_t size;  // elements, and whether all its arrays are aligned for four at once
    void* at[kPtrs];
  };
  Slot t[kMost];
  uint32_t first[kMost + 1];  // each tensor's first chunk; the last: how many there are
  int n;
  AdamWStep s;
  void add(const AdamWTensor& q, uint32_t chunks) {
    Slot& x = t[n];
    x.size = static_cast<uint64_t>(q.n) << 1 | q.wide;
    x.at[0] = q.p;
    x.at[1] = const_cast<void*>(q.g);
    x.at[2] = q.m;
    x.at[3] = q.v;
    if constexpr (P == kMaster) x.at[4] = q.master;
    if constexpr (B8) {
      x.at[kPtrs - 2] = q.m_scales;
      x.at[kPtrs - 1] = q.v_scales;
    }
    first[n + 1] = first[n] + chunks;
    ++n;
  }
  __device__ __forceinline__ AdamWTensor get(int i) const {
    const Slot& x = t[i];
    AdamWTensor q{};
    q.n = static_cast<int64_t>(x.size >> 1);
    q.wide = x.size & 1;
    q.p = x.at[0];
    q.g = x.at[1];
    q.m = x.at[2];
    q.v = x.at[3];
    if constexpr (P == kMaster) q.master = x.at[4];
    if constexpr (B8) {
      q.m_scales = static_cast<float*>(x.at[kPtrs - 2]);
      q.v_scales = static_cast<float*>(x.at[kPtrs - 1]);
    }
    return q;
  }
};

__device__ __forceinline__ float two_to(int n) {
  return __uint_as_float(static_cast<uint32_t>(n + 127) << 23);
}
__device__ __forceinline__ bool finite(float v) {
  return (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u;
}

// Elements i .. i + 3 of an array of n.  WHOLE: all of them are there, and the
// address is aligned for one access.
template <bool WHOLE, class T>
__device__ __forceinline__ void load4(const T* p, int64_t i, int64_t n, T (&v)[kV]) {
  struct alignas(sizeof(T) * kV) Pack {
    T v[kV];
  };
  if constexpr (WHOLE) {
    const Pack q = *reinterpret_cast<const Pack*>(p + i);
#pragma unroll
    for (int j = 0; j < kV; ++j) v[j] = q.v[j];
  } else {
#pragma unroll
    for (int j = 0; j < kV; ++j) v[j] = i + j < n ? p[i + j] : T(0);
  }
}
template <bool WHOLE, class T>
__device__ __forceinline__ void store4(T* p, int64_t i, int64_t n, const T (&v)[kV]) {
  struct alignas(sizeof(T) * kV) Pack {
    T v[kV];
  };
  if constexpr (WHOLE) {
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

// Bits of h spread over all 32: two products with odd numbers, shifts between.
__host__ __device__ constexpr uint32_t mix(uint32_t h) {
  h = (h ^ (h >> 16)) * 0x6A09E667u;
  h = (h ^ (h >> 15)) * 0x9E3779B9u;
  return h ^ (h >> 16);
}
// Two numbers in (0, 1), 16 bits and a half each: of m's code, of v's.
struct Draw {
  float m, v;
};
__device__ __forceinline__ Draw draw(uint32_t h) {
  return {(static_cast<float>(h & 0xFFFFu) + 0.5f) * 0x1p-16f,
          (static_cast<float>(h >> 16) + 0.5f) * 0x1p-16f};
}

// The e4m3 value next to a (|a| <= 448) below it or above, so that a is the mean
// over u: |a| in places of its binade, at least 2^-9 each.
__device__ __forceinline__ float e4m3_mean(float a, float u) {
  const int e = max(static_cast<int>(__float_as_uint(a) >> 23 & 0xFFu) - 127, -6) - 3;
  return copysignf(floorf(fabsf(a) * two_to(-e) + u) * two_to(e), a);
}

// Exponent n of the smallest scale 2^n >= 2^-126 with top <= limit * 2^n, limit =
// 1.mant * 2^log: 0 for a top of zero.
__device__ __forceinline__ int scale_exponent(uint32_t top, uint32_t mant, int log) {
  if (top == 0u) return 0;
  const int e = static_cast<int>(top >> 23) - 127;
  return max(-126, (top & 0x7FFFFFu) <= mant ? e - log : e - log + 1);
}

// What a lane holds of a block before its update.
struct Loaded {
  float p32[kV];
  uint16_t p16[kV], g16[kV];
  float g32[kV], m32[kV], v32[kV];
  uint8_t mc[kV], vc[kV];
  float ms, vs;
};

// The block from element `from` on.  key: the step's, for the hash.
template <int M, int P, bool GBF16, bool WHOLE>
__device__ __forceinline__ void update(const AdamWTensor& q, const AdamWStep& h, float size,
                                       float root, float gs, uint32_t key, int64_t from, int lane) {
  constexpr bool B8 = M != kFloats;
  const int64_t n = q.n;
  const int64_t i = from + lane * kV, blk = from / kBlock;
  Loaded x;
  bool marked = false;  // the block holds a root that is not finite
  if (P == kF32) load4<WHOLE>(static_cast<const float*>(q.p), i, n, x.p32);
  if (P == kBf16) load4<WHOLE>(static_cast<const uint16_t*>(q.p), i, n, x.p16);
  if (P == kMaster) load4<WHOLE>(static_cast<const float*>(q.master), i, n, x.p32);
  if (GBF16)
    load4<WHOLE>(static_cast<const uint16_t*>(q.g), i, n, x.g16);
  else
    load4<WHOLE>(static_cast<const float*>(q.g), i, n, x.g32);
  if (B8) {
    load4<WHOLE>(static_cast<const uint8_t*>(q.m), i, n, x.mc);
    load4<WHOLE>(static_cast<const uint8_t*>(q.v), i, n, x.vc);
    x.ms = q.m_scales[blk];
    x.vs = q.v_scales[blk];
    marked = !(x.vs == x.vs);
    const uint32_t e = __float_as_uint(x.vs) & 0xFFu;
    if (marked && e != 0u) x.vs = __uint_as_float(e << 23);
  } else {
    load4<WHOLE>(static_cast<const float*>(q.m), i, n, x.m32);
    load4<WHOLE>(static_cast<const float*>(q.v), i, n, x.v32);
  }
  float m[kV], v[kV], r[kV], p[kV];
  if (B8) {
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < kV; ++j) w |= static_cast<uint32_t>(x.mc[j]) << (8 * j);
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
    m[0] = lo[0] * x.ms; m[1] = lo[1] * x.ms;
    m[2] = hi[0] * x.ms; m[3] = hi[1] * x.ms;
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const int code = x.vc[j], e = max((code >> 5) - 1, 0);
      const float s = static_cast<float>((code - 32 * e) << e) * x.vs;
      v[j] = marked && code == 255 ? __builtin_inff() : s * s;
    }
  } else {
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      m[j] = x.m32[j];
      v[j] = x.v32[j];
    }
  }
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    float g = GBF16 ? bf16_to_f32(x.g16[j]) : x.g32[j];
    g = g * gs;
    m[j] = m[j] * h.beta1 + g * h.rest1;
    v[j] = v[j] * h.beta2 + g * g * h.rest2;
    r[j] = sqrtf(v[j]);
    p[j] = P == kBf16 ? bf16_to_f32(x.p16[j]) : x.p32[j];
    p[j] = p[j] * h.keep - m[j] / (r[j] * root + h.eps) * size;
  }
  if (P != kF32) {
    uint16_t half[kV];
#pragma unroll
    for (int j = 0; j < kV; ++j) half[j] = f32_to_bf16(p[j]);
    store4<WHOLE>(static_cast<uint16_t*>(q.p), i, n, half);
  }
  if (P != kBf16) store4<WHOLE>(static_cast<float*>(P == kMaster ? q.master : q.p), i, n, p);
  if (B8) {
    uint32_t top_m, top_r;
    auto tops = [&](auto counts) {
      top_m = top_r = 0;
#pragma unroll
      for (int j = 0; j < kV; ++j)
        if ((WHOLE || i + j < n) && counts(j)) {
          if (finite(m[j])) top_m = max(top_m, __float_as_uint(m[j]) & 0x7FFFFFFFu);
          top_r = max(top_r, __float_as_uint(r[j]) & 0x7FFFFFFFu);
        }
      top_m = wave_max_u32(top_m);
      top_r = wave_max_u32(top_r);
    };
    tops([](int) { return true; });
    const bool odd = top_r >= 0x7F800000u;
    if (odd) tops([&](int j) { return finite(r[j]); });
    const int em = scale_exponent(top_m, 0x600000u, 8);   // 448 = 1.75 * 2^8
    // 4032 = 1.96875 * 2^11, or below code 255: 3968 = 1.9375 * 2^11
    const int er = scale_exponent(top_r, odd ? 0x780000u : 0x7C0000u, 11);
    const float im = two_to(-em), ir = two_to(-er);
    uint8_t mc[kV], vc[kV];
    float a[kV];
    const uint32_t place = M == kHashed ? static_cast<uint32_t>(i) +
                                              mix(key + static_cast<uint32_t>(from >> 32))
                                        : 0u;
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      a[j] = finite(m[j]) ? m[j] * im : __uint_as_float(0x7FC00000u);
      const float s = fminf(r[j] * ir, 4032.0f);  // a number where r is none, too
      const int e = max(static_cast<int>(__float_as_uint(s) >> 23) - 126 - 6, 0);
      const float t = s * two_to(-e);
      int code = 32 * e;
      if constexpr (M == kHashed) {
        const Draw u = draw(mix(place + j));
        if (finite(m[j])) a[j] = e4m3_mean(a[j], u.m);
        // t^2 as the mean of low^2 and (low + 1)^2
        const float low = floorf(t);
        code += static_cast<int>(low) + ((t - low) * (t + low) > u.v * (2.0f * low + 1.0f));
      } else {
        code += static_cast<int>(rintf(t));
      }
      vc[j] = static_cast<uint8_t>(r[j] > 0.0f ? max(code, 1) : code);
    }
    int w = 0;
    w = __builtin_amdgcn_cvt_pk_fp8_f32(a[0], a[1], w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(a[2], a[3], w, true);
#pragma unroll
    for (int j = 0; j < kV; ++j) mc[j] = static_cast<uint8_t>(w >> (8 * j));
    if (odd) {
#pragma unroll
      for (int j = 0; j < kV; ++j)
        if (!finite(r[j])) {
          vc[j] = 255;
          // m moves nothing there; 0x7E is 448
          if (finite(m[j]) && !(fabsf(m[j] * im) <= 448.0f)) mc[j] = m[j] < 0.0f ? 0xFE : 0x7E;
        }
    }
    store4<WHOLE>(static_cast<uint8_t*>(q.m), i, n, mc);
    store4<WHOLE>(static_cast<uint8_t*>(q.v), i, n, vc);
    if (lane == 0) {
      q.m_scales[blk] = two_to(em);
      q.v_scales[blk] = odd ? __uint_as_float(0x7FC00000u | static_cast<uint32_t>(er + 127))
                            : two_to(er);
    }
  } else {
    store4<WHOLE>(static_cast<float*>(q.m), i, n, m);
    store4<WHOLE>(static_cast<float*>(q.v), i, n, v);
  }
}

template <int M, int P, bool GBF16>
__global__ __launch_bounds__(kThreads) void adamw_step(const Batch<M != kFloats, P> b) {
  static_assert(sizeof(b) <= 4096, "a launch's arguments");
  const int lane = threadIdx.x & (kWave - 1);
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t my_first = b.first[min(lane, b.n)];
  const uint32_t chunks = b.first[b.n];
  const int64_t step = max(*b.s.step, int64_t(1));
  const double t = static_cast<double>(step);
  const uint32_t key = mix(static_cast<uint32_t>(step) + mix(static_cast<uint32_t>(step >> 32)));
  const float size = static_cast<float>(b.s.lr / (1.0 - exp(t * b.s.log_beta1)));
  const float root = static_cast<float>(1.0 / sqrt(1.0 - exp(t * b.s.log_beta2)));
  const float gs = b.s.grad_scale ? *b.s.grad_scale : 1.0f;
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    // the last tensor whose first chunk is not behind c
    const int at = __popcll(__ballot(lane < b.n && my_first <= c)) - 1;
    const AdamWTensor q = b.get(at);
    const int64_t from = (static_cast<int64_t>(c - b.first[at]) * kWaves + wv) * kBlock;
    if (q.wide && from + kBlock <= q.n)
      update<M, P, GBF16, true>(q, b.s, size, root, gs, key, from, lane);
    else if (from < q.n)
      update<M, P, GBF16, false>(q, b.s, size, root, gs, key, from, lane);
  }
}

// How a tensor is held and its codes are rounded, as a number.
constexpr int kKinds = 18;
constexpr int kind_of(int moments, int store, bool gbf16) { return (moments * 3 + store) * 2 + gbf16; }
int kind_of(const AdamWTensor& t, bool nearest) {
  return kind_of(!t.m_scales ? kFloats : nearest ? kNearest : kHashed,
                 t.master ? kMaster : t.p_bf16 ? kBf16 : kF32, t.g_bf16);
}

// The tensors of one kind, a batch of them a launch.
template <int KIND>
hipError_t go(const AdamWSource& src, int n, const AdamWStep& s, hipStream_t stream) {
  constexpr bool GBF16 = KIND % 2;
  constexpr int M = KIND / 6, P = KIND / 2 % 3;
  static_assert(KIND == kind_of(M, P, GBF16));
  constexpr int64_t per = kWaves * kBlock;
  Batch<M != kFloats, P> b;
  b.n = 0;
  b.first[0] = 0;
  b.s = s;
  auto flush = [&]() -> hipError_t {
    if (b.n == 0) return hipSuccess;
    const uint32_t chunks = b.first[b.n];
    const dim3 grid(chunks < kMaxGrid ? chunks : kMaxGrid), block(kThreads);
    const hipError_t e = launch(adamw_step<M, P, GBF16>, grid, block, 0, stream, b);
    b.n = 0;
    return e;
  };
  for (int i = 0; i < n; ++i) {
    const AdamWTensor t = src.get(src.tensors, i);
    if (t.n == 0 || kind_of(t, s.nearest) != KIND) continue;
    const int64_t chunks = (t.n + per - 1) / per;
    if (b.n == b.kMost || (b.n > 0 && b.first[b.n] + chunks > INT32_MAX)) {
      const hipError_t e = flush();
      if (e != hipSuccess) return e;
    }
    b.add(t, static_cast<uint32_t>(chunks));
  }
  return flush();
}
template <int... KIND>
hipError_t go_each(uint32_t present, const AdamWSource& src, int n, const AdamWStep& s,
                   hipStream_t stream, std::integer_sequence<int, KIND...>) {
  hipError_t e = hipSuccess;
  ((present >> KIND & 1 && e == hipSuccess ? void(e = go<KIND>(src, n, s, stream)) : void()), ...);
  return e;
}

}  // namespace

// Tensors of one kind share launches.
hipError_t launch_adamw(const AdamWSource& src, int n, const AdamWStep& s, hipStream_t stream) {
  uint32_t present = 0;
  for (int i = 0; i < n; ++i) {
    const AdamWTensor t = src.get(src.tensors, i);
    if (t.n != 0) present |= 1u << kind_of(t, s.nearest);
  }
  return go_each(present, src, n, s, stream, std::make_integer_sequence<int, kKinds>{});
}

}  // namespace moe
