// The whole layer for a few tokens in two kernels, on bf16 experts, e4m3 codes
// with a float32 scale per 128 x 128, or 8-bit integers with one per output
// channel.  With s a (token, expert) pair of the routing and e its expert:
//   few_gate_up   h[s] = silu(G_e x[t]) * (U_e x[t])
//   few_down      out[t] = sum_j w[t][j] D_e h[t k + j]  (+ D h of the shared expert)
//
// Bound by reading the hit experts' weights once.  Neither kernel needs the
// tokens grouped beforehand: a workgroup sets a bit per chosen expert in LDS,
// takes its expert from the set bits and finds the expert's pairs by ballots
// over the (at most 256) ids.  A second kernel is needed since every element of
// out wants all of h; combining there spares y's way through memory and a launch.
//
// The weights go from memory straight into the matrix instruction's A side, 16
// of its rows x 64 bytes a load: there is nothing to share through LDS, so the
// loads need no barrier.  The tokens are the B side, up to 16 a fragment and two
// fragments at once; lanes without a token multiply zeros, which no one reads.
// Codes are widened to bf16, which holds each of them exactly.  x is not
// quantised; h is kept as two bf16 values (16 significant bits, off by 2^-17 at
// most, the second one's product costing little beside the weights' bytes).
// All sums are float32, in an order that depends on the sizes and the number of
// experts hit alone.
#include <type_traits>

#include "common.h"
#include "launch.h"

#pragma clang fp contract(off)  // the fused multiply-adds are written out

namespace moe {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kCols = 16;     // weight rows (output columns) of a fragment
constexpr int kBlock = 128;   // rows and columns per scale of e4m3 codes
constexpr int kMaxPairs = 256, kMaxIds = 1024;
constexpr int kIds = kMaxPairs / kWave;  // ids a lane holds
constexpr int kChunkRows = 32;           // tokens per pass over an expert's weights

template <int KIND>
struct Fmt {
  static constexpr int kElem = KIND == kFewBf16 ? 2 : 1;
  static constexpr int kChunk = 16 / kElem;       // values a lane loads at once
  static constexpr int kStep = 4 * kChunk;        // contraction of one load
  static constexpr int kLoads = 4;                // loads of a turn
  static constexpr int kTurn = kLoads * kStep;    // contraction of a turn
};

// The pairs' ids, a few per lane; -1 where there is none or it names no expert.
struct Ids {
  int id[kIds];
};
__device__ __forceinline__ Ids load_ids(const FewLayer& g, int lane) {
  Ids r;
#pragma unroll
  for (int i = 0; i < kIds; ++i) {
    const int s = lane + i * kWave;
    const int v = s < g.T * g.k ? g.topk_idx[s] : -1;
    r.id[i] = v >= 0 && v < g.E ? v : -1;
  }
  return r;
}

// One bit per expert hit; every thread of the workgroup calls it.
__device__ __forceinline__ void mark_experts(const Ids& ids, uint32_t* bits) {
  const int t = threadIdx.x;
  if (t < kMaxIds / 32) bits[t] = 0u;
  __syncthreads();
  if (t < kWave) {
#pragma unroll
    for (int i = 0; i < kIds; ++i)
      if (ids.id[i] >= 0) atomicOr(&bits[ids.id[i] >> 5], 1u << (ids.id[i] & 31));
  }
  __syncthreads();
}

// Inclusive sum over the lower 32 lanes (each half of the wavefront for itself).
__device__ __forceinline__ int scan32(int v, int lane) {
  for (int off = 1; off < 32; off <<= 1) {
    const int u = __shfl_up(v, off, 32);
    if ((lane & 31) >= off) v += u;
  }
  return v;
}

// The expert of the n-th set bit, -1 past the last (a wavefront together).
__device__ __forceinline__ int nth_expert(const uint32_t* bits, int n, int lane) {
  uint32_t m = bits[lane & 31];
  const int c = __popc(m), inc = scan32(c, lane), first = inc - c;
  const bool here = lane < 32 && n >= first && n < inc;
  const uint64_t who = __ballot(here);
  if (!who) return -1;
  int e = 0;
  if (here) {
    for (int i = n - first; i > 0; --i) m &= m - 1;
    e = lane * 32 + __ffs(m) - 1;
  }
  return __builtin_amdgcn_readlane(e, __ffsll(static_cast<unsigned long long>(who)) - 1);
}

// The pairs of expert e, ascending, into list; returns how many (a wavefront
// together; its own list).
__device__ __forceinline__ int pairs_of(const Ids& ids, int e, int lane, uint8_t* list) {
  const uint64_t lower = (1ull << lane) - 1ull;
  int n = 0;
#pragma unroll
  for (int i = 0; i < kIds; ++i) {
    const uint64_t m = __ballot(ids.id[i] == e);
    if (ids.id[i] == e) list[n + __popcll(m & lower)] = static_cast<uint8_t>(lane + i * kWave);
    n += __popcll(m);
  }
  // the other lanes' entries before this one reads them
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  return n;
}

// Eight codes as bf16, exactly.
template <int KIND>
__device__ __forceinline__ bf16x8_t widen(uint32_t lo, uint32_t hi) {
  if constexpr (KIND == kFewE4m3) {
    const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  } else {
    bf16x8_t r;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t w = j < 4 ? lo : hi;
      r[j] = static_cast<__bf16>(
          static_cast<float>(static_cast<int8_t>((w >> (8 * (j & 3))) & 0xFFu)));
    }
    return r;
  }
}

__device__ __forceinline__ u32x4_t load16(const void* p, int64_t byte) {
  return *reinterpret_cast<const u32x4_t*>(static_cast<const uint8_t*>(p) + byte);
}

__device__ __forceinline__ f32x4_t mma(bf16x8_t w, u32x4_t x, f32x4_t acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8_t, x), acc, 0, 0, 0);
}

// The B side: this lane's row of x (or of h's two parts) in each fragment.
template <int NB, bool SPLIT>
struct Rows {
  const uint16_t* hi[NB];
  const uint16_t* lo[NB];
  bool on[NB];
  __device__ __forceinline__ f32x4_t product(bf16x8_t w, int b, int k, f32x4_t acc) const {
    u32x4_t v{0, 0, 0, 0}, u{0, 0, 0, 0};
    if (on[b]) {
      v = load16(hi[b] + k, 0);
      if constexpr (SPLIT) u = load16(lo[b] + k, 0);
    }
    acc = mma(w, v, acc);
    if constexpr (SPLIT) acc = mma(w, u, acc);
    return acc;
  }
};

// One turn of the contraction, [k0, k0 + kTurn): this wavefront's 16 weight rows
// (wp: the lane's row, its part of a load) times the tokens.  scales: of the
// turn's blocks of 128 (e4m3).
template <int KIND, int NB, bool SPLIT>
__device__ __forceinline__ void turn(const uint8_t* wp, const float* scales, int k0, int K, int q,
                                     const Rows<NB, SPLIT>& rows, f32x4_t (&acc)[NB]) {
  using F = Fmt<KIND>;
  u32x4_t w[F::kLoads];
#pragma unroll
  for (int u = 0; u < F::kLoads; ++u)
    w[u] = k0 + u * F::kStep < K ? load16(wp, static_cast<int64_t>(k0 + u * F::kStep) * F::kElem)
                                 : u32x4_t{0, 0, 0, 0};
  if constexpr (KIND == kFewBf16) {
#pragma unroll
    for (int u = 0; u < F::kLoads; ++u) {
      const int k = k0 + u * F::kStep;
      if (k >= K) break;
#pragma unroll
      for (int b = 0; b < NB; ++b)
        acc[b] = rows.product(__builtin_bit_cast(bf16x8_t, w[u]), b, k + q * F::kChunk, acc[b]);
    }
  } else {
    constexpr int kPer = kBlock / F::kStep;  // loads per block
#pragma unroll
    for (int h = 0; h < F::kLoads; h += kPer) {
      if (k0 + h * F::kStep >= K) break;
      f32x4_t p[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) p[b] = KIND == kFewE4m3 ? f32x4_t{0, 0, 0, 0} : acc[b];
#pragma unroll
      for (int u = h; u < h + kPer; ++u) {
        const int k = k0 + u * F::kStep;
        if (k >= K) break;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const bf16x8_t c = widen<KIND>(w[u][2 * v], w[u][2 * v + 1]);
#pragma unroll
          for (int b = 0; b < NB; ++b)
            p[b] = rows.product(c, b, k + q * F::kChunk + v * 8, p[b]);
        }
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if constexpr (KIND == kFewE4m3) {
          const float s = scales[(k0 + h * F::kStep) / kBlock];
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[b][j] = fmaf(s, p[b][j], acc[b][j]);
        } else {
          acc[b] = p[b];
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// gate and up: a workgroup takes 16 columns of one expert's h; four wavefronts
// the gate's rows and four the up's, in turns along the contraction.
// ---------------------------------------------------------------------------
constexpr int kGuWaves = 8, kGuThreads = kGuWaves * kWave;

template <int KIND>
__global__ __launch_bounds__(kGuThreads) void few_gate_up(FewLayer g, int tiles) {
  using F = Fmt<KIND>;
  __shared__ float part[kGuWaves][kChunkRows][kCols + 1];
  __shared__ uint32_t bits[kMaxIds / 32];
  __shared__ uint8_t lists[kGuWaves][kMaxPairs];
  const int t = threadIdx.x, lane = t & (kWave - 1);
  const int wv = __builtin_amdgcn_readfirstlane(t / kWave);
  const int n0 = static_cast<int>(blockIdx.x) % tiles * kCols;
  int slot = static_cast<int>(blockIdx.x) / tiles;
  const bool shared = g.shared && slot == 0;
  slot -= g.shared;
  int e = 0, n = g.T;
  const uint8_t* list = lists[wv];
  if (!shared) {
    const Ids ids = load_ids(g, lane);
    mark_experts(ids, bits);
    e = nth_expert(bits, slot, lane);
    if (e < 0) return;
    n = pairs_of(ids, e, lane, lists[wv]);
  }
  const int i16 = lane & 15, q = lane >> 4;
  const int row0 = (wv < kGuWaves / 2 ? 0 : g.f) + n0;  // of this wavefront's weight rows
  const uint8_t* wbase = static_cast<const uint8_t*>(shared ? g.shared_gate_up : g.gate_up);
  const float* sbase = shared ? g.shared_gate_up_scales : g.gate_up_scales;
  const uint8_t* wp = wbase +
                      (static_cast<int64_t>(e) * 2 * g.f + row0 + i16) * g.d * F::kElem + q * 16;
  const float* ws = nullptr;
  if (KIND == kFewE4m3)
    ws = sbase + (static_cast<int64_t>(e) * ((2 * g.f + kBlock - 1) / kBlock) + row0 / kBlock) *
                     ((g.d + kBlock - 1) / kBlock);
  const uint16_t* x = static_cast<const uint16_t*>(g.x);
  for (int m0 = 0; m0 < n; m0 += kChunkRows) {
    auto pass = [&](auto nb) {
      constexpr int NB = decltype(nb)::value;
      Rows<NB, false> rows;
      f32x4_t acc[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int r = m0 + b * 16 + i16;
        rows.on[b] = r < n;
        const int token = r >= n ? 0 : shared ? r : list[r] / g.k;
        rows.hi[b] = x + static_cast<int64_t>(token) * g.d;
        acc[b] = f32x4_t{0, 0, 0, 0};
      }
      for (int k0 = (wv & 3) * F::kTurn; k0 < g.d; k0 += 4 * F::kTurn)
        turn<KIND, NB, false>(wp, ws, k0, g.d, q, rows, acc);
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) part[wv][b * 16 + i16][q * 4 + j] = acc[b][j];
    };
    if (n - m0 > 16)
      pass(std::integral_constant<int, 2>{});
    else
      pass(std::integral_constant<int, 1>{});
    __syncthreads();
    const int r = t / kCols, c = t % kCols;  // 512 threads: 32 rows of 16 columns
    if (m0 + r < n) {
      float gate = 0.0f, up = 0.0f;
#pragma unroll
      for (int w = 0; w < kGuWaves / 2; ++w) {
        gate += part[w][r][c];
        up += part[w + kGuWaves / 2][r][c];
      }
      if (KIND == kFewInt8) {
        const float* s = sbase + static_cast<int64_t>(e) * 2 * g.f + n0 + c;
        gate *= s[0];
        up *= s[g.f];
      }
      const float h = silu(gate) * up;
      const uint16_t hi = f32_to_bf16(h);
      const float rest = h - bf16_to_f32(hi);
      // an infinity has no rest
      const uint16_t lo = rest == rest ? f32_to_bf16(rest) : static_cast<uint16_t>(0);
      const int row = shared ? g.T * g.k + m0 + r : list[m0 + r];
      const int64_t at = static_cast<int64_t>(row) * g.f + n0 + c;
      g.h_hi[at] = hi;
      g.h_lo[at] = lo;
    }
    __syncthreads();
  }
}
static_assert(kGuThreads == kChunkRows * kCols, "a thread per element of h");

// ---------------------------------------------------------------------------
// down and combine: a workgroup takes 16 columns of out.  Its units of work are
// (expert hit, part of the contraction), dealt to its wavefronts in turn; each
// leaves its rows' sums in LDS, which one meeting later are weighted and added
// up in the pairs' order.
// ---------------------------------------------------------------------------
constexpr int kDnWaves = 16, kDnThreads = kDnWaves * kWave;
constexpr int kSumRows = 576;  // rows of sums in LDS: the pairs' and the tokens', per part
constexpr int kUnits = 128;    // units to have, so that the wavefronts get about as many each

template <int KIND>
__global__ __launch_bounds__(kDnThreads) void few_down(FewLayer g) {
  using F = Fmt<KIND>;
  __shared__ float sums[kSumRows][kCols + 4];
  __shared__ uint32_t bits[kMaxIds / 32];
  __shared__ uint16_t active[kMaxPairs];
  __shared__ uint8_t lists[kDnWaves][kMaxPairs];
  __shared__ int n_active;
  const int t = threadIdx.x, lane = t & (kWave - 1);
  const int wv = __builtin_amdgcn_readfirstlane(t / kWave);
  const int n0 = static_cast<int>(blockIdx.x) * kCols;
  const Ids ids = load_ids(g, lane);
  mark_experts(ids, bits);
  if (wv == 0) {
    uint32_t m = lane < 32 ? bits[lane] : 0u;
    const int c = __popc(m), inc = scan32(c, lane);
    for (int at = inc - c; m; m &= m - 1)
      active[at++] = static_cast<uint16_t>(lane * 32 + __ffs(m) - 1);
    if (lane == 31) n_active = inc;
  }
  __syncthreads();
  const int pairs = g.T * g.k, n_rows = pairs + (g.shared ? g.T : 0);
  const int groups = n_active + g.shared;
  const int turns = (g.f + F::kTurn - 1) / F::kTurn;
  int parts = 1;
  while (groups * parts < kUnits && 2 * parts <= turns && 2 * parts * n_rows <= kSumRows) parts *= 2;
  const int i16 = lane & 15, q = lane >> 4;
  for (int unit = wv; unit < groups * parts; unit += kDnWaves) {
    const int grp = unit / parts, part = unit - grp * parts;
    const bool shared = g.shared && grp == 0;
    int e = 0, n = g.T;
    if (!shared) {
      e = active[grp - g.shared];
      n = pairs_of(ids, e, lane, lists[wv]);
    }
    const int from = part * turns / parts * F::kTurn;
    const int to = min(g.f, (part + 1) * turns / parts * F::kTurn);
    const uint8_t* wbase = static_cast<const uint8_t*>(shared ? g.shared_down : g.down);
    const float* sbase = shared ? g.shared_down_scales : g.down_scales;
    const uint8_t* wp =
        wbase + (static_cast<int64_t>(e) * g.d + n0 + i16) * g.f * F::kElem + q * 16;
    const float* ws = nullptr;
    if (KIND == kFewE4m3)
      ws = sbase + (static_cast<int64_t>(e) * ((g.d + kBlock - 1) / kBlock) + n0 / kBlock) *
                       ((g.f + kBlock - 1) / kBlock);
    for (int m0 = 0; m0 < n; m0 += kChunkRows) {
      auto pass = [&](auto nb) {
        constexpr int NB = decltype(nb)::value;
        Rows<NB, true> rows;
        f32x4_t acc[NB];
        int row[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const int r = m0 + b * 16 + i16;
          rows.on[b] = r < n;
          row[b] = r >= n ? 0 : shared ? pairs + r : lists[wv][r];
          rows.hi[b] = g.h_hi + static_cast<int64_t>(row[b]) * g.f;
          rows.lo[b] = g.h_lo + static_cast<int64_t>(row[b]) * g.f;
          acc[b] = f32x4_t{0, 0, 0, 0};
        }
        for (int k0 = from; k0 < to; k0 += F::kTurn)
          turn<KIND, NB, true>(wp, ws, k0, to, q, rows, acc);
        f32x4_t s{1, 1, 1, 1};
        if constexpr (KIND == kFewInt8)
          s = *reinterpret_cast<const f32x4_t*>(sbase + static_cast<int64_t>(e) * g.d + n0 + q * 4);
#pragma unroll
        for (int b = 0; b < NB; ++b)
          if (rows.on[b])
            *reinterpret_cast<f32x4_t*>(&sums[part * n_rows + row[b]][q * 4]) = acc[b] * s;
      };
      if (n - m0 > 16)
        pass(std::integral_constant<int, 2>{});
      else
        pass(std::integral_constant<int, 1>{});
    }
  }
  __syncthreads();
  for (int o = t; o < g.T * kCols; o += kDnThreads) {
    const int tok = o / kCols, c = o % kCols;
    float v = 0.0f;
    auto whole = [&](int row) {
      float y = sums[row][c];
      for (int p = 1; p < parts; ++p) y += sums[p * n_rows + row][c];
      return y;
    };
    for (int j = 0; j < g.k; ++j) {
      const int s = tok * g.k + j, id = g.topk_idx[s];
      if (id >= 0 && id < g.E) v = fmaf(g.topk_w[s], whole(s), v);
    }
    if (g.shared) v += whole(pairs + tok);
    const int64_t at = static_cast<int64_t>(tok) * g.d + n0 + c;
    if (g.out_f32)
      static_cast<float*>(g.out)[at] = v;
    else
      static_cast<uint16_t*>(g.out)[at] = f32_to_bf16(v);
  }
}

template <int KIND>
hipError_t go(const FewLayer& g, hipStream_t stream) {
  const int pairs = g.T * g.k, tiles = g.f / kCols;
  const int slots = (pairs < g.E ? pairs : g.E) + g.shared;
  const hipError_t e = launch(few_gate_up<KIND>, dim3(static_cast<uint32_t>(slots * tiles)),
                              dim3(kGuThreads), 0, stream, g, tiles);
  if (e != hipSuccess) return e;
  return launch(few_down<KIND>, dim3(static_cast<uint32_t>(g.d / kCols)), dim3(kDnThreads), 0,
                stream, g);
}

}  // namespace

size_t few_workspace(int T, int k, int f, bool shared) {
  return static_cast<size_t>(T) * (k + shared) * f * 2 * sizeof(uint16_t);
}

hipError_t launch_layer_few(const FewLayer& g, FewKind kind, hipStream_t stream) {
  switch (kind) {
    case kFewBf16: return go<kFewBf16>(g, stream);
    case kFewE4m3: return go<kFewE4m3>(g, stream);
    default: return go<kFewInt8>(g, stream);
  }
}

}  // namespace moe
