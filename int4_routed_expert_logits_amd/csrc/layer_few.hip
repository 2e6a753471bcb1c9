// The whole layer for a few tokens in two kernels (and one that joins the sums of
// workgroups that share a narrow out's steps), on bf16 experts, e4m3 codes
// with a float32 scale per 128 x 128, or 8-bit integers with one per output
// channel.  With s a (token, expert) pair of the routing and e its expert:
//   few_gate_up   h[s] = silu(G_e x[t]) * (U_e x[t])
//   few_down      out[t] = sum_j w[t][j] D_e h[t k + j]  (+ D h of the shared expert)
//
// Bound by reading the hit experts' weights once.  few_gate_up does not need the
// tokens grouped beforehand: a workgroup sets a bit per chosen expert in LDS,
// takes its expert from the set bits and finds the expert's pairs by ballots
// over the (at most 256) ids; one more workgroup writes that grouping down for
// few_down.  A second kernel is needed since every element of out wants all of h;
// combining there spares y's way through memory and a launch.
//
// The weights go from memory straight into the matrix instruction's A side, 8 of
// its rows x 128 bytes a load: there is nothing to share through LDS, so the loads
// need no barrier.  The tokens are the B side, up to 8 a fragment and two
// fragments at once.  Codes are widened to bf16, which holds each of them exactly.
// x is not quantised; h is kept as a sum of bf16 values: three hold all of its 24
// bits, and two (17 bits) do for an out of bf16, whose own rounding is 2^-9.
// All sums are float32, in an order that depends on the sizes and the routing
// alone.
//
// Measured (the kernels' own times under the profiler, which runs some per cent
// slower): one token over 8 of 256 bf16 experts of 6144 x 2048 and a shared one 134 us
// with its routing, 80 (453 MB, 5.7 TB/s) and 43 us (226 MB, 5.3 TB/s); 8 tokens on
// integers 373-388, 253 (1.47 GB, 5.8 TB/s) and 134 us (0.74 GB, 5.5 TB/s); 32 tokens
// over 64 bf16 experts of 2048 x 1024 159-162, 96 (537 MB, 5.6 TB/s) and 54 us (268 MB,
// 4.9 TB/s beside what is read of h); 3 tokens routed to 23 e4m3 experts of 2048 x 512
// 25, 12.5 (50 MB) and 12.7 us (25 MB), each a workgroup's few steps and their latency.
// Steps that got there, for the first two: 16 weight rows x 64 bytes a load and
// tokens by masked loads 188 / 633, 8 rows x 128 bytes without masks 145 / 726, gate
// and up (or two column tiles) sharing their tokens, one step at a time with the
// next weights under way 157 / 467, few_down's steps shared evenly and the
// grouping handed on 145 / 455, its columns by the CUs 136 / 405, neighbouring lanes reading 32 bytes
// together, where each had read 16 of another row and the cache took an access for
// every lane, 134 / 385.  Two or more steps at a time, or the tokens a step ahead as
// well, gain nothing and need the registers; several tiles of h a workgroup cost
// 2 to 4% in short calls and gain 4% on e4m3 in long ones; a second workgroup per CU
// of few_down costs 2 to 7%.
#include <type_traits>

#include "common.h"
#include "launch.h"

#pragma clang fp contract(off)  // the fused multiply-adds are written out

namespace moe {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kCols = 8;      // weight rows (output columns) of a fragment
constexpr int kBlock = 128;   // rows and columns per scale of e4m3 codes
constexpr int kMaxPairs = 256, kMaxIds = 1024, kCus = 256;
constexpr int kIds = kMaxPairs / kWave;  // ids a lane holds

// A load of a wavefront: 8 weight rows x 128 bytes.  The matrix instruction's 16
// rows are those 8 with the even 16-byte chunks and again with the odd ones, its
// 16 columns 8 tokens with the one and with the other chunks of x, so that on its
// result's diagonal lie 8 x 8 times both parts' sums.  Neighbouring lanes hold the
// two parts, so that they read 32 bytes together.
struct Lane {
  int row, part, q;  // of 8 rows or tokens, of 2 chunks, of 4 pairs of chunks
  int tail;          // 1: in the second 64 bytes of a load
  __device__ __forceinline__ explicit Lane(int lane)
      : row((lane >> 1) & 7), part(lane & 1), q(lane >> 4), tail(lane >> 5) {}
  __device__ __forceinline__ int chunk() const { return q * 2 + part; }
};
template <int KIND>
struct Fmt {
  static constexpr int kElem = KIND == kFewBf16 ? 2 : 1;
  static constexpr int kChunk = 16 / kElem;  // values a lane loads at once
  static constexpr int kHalf = 4 * kChunk;   // contraction of half a load
  static constexpr int kStep = 2 * kHalf;    // ... of a load
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

// The grouping as few_gate_up leaves it for few_down: the experts hit, ascending,
// and each one's pairs, ascending.
struct alignas(16) FewTable {
  int32_t n;                           // experts hit
  int32_t most;                        // pairs of the one that has most
  uint16_t active[kMaxPairs];          // the experts
  uint16_t start[kMaxPairs + 8];       // where an expert's pairs begin in `pair`; the end
  uint8_t pair[kMaxPairs];
  uint8_t group[kMaxPairs];            // of a pair: which of `active`,
  uint8_t rank[kMaxPairs];             // the how many-th of its pairs,
  uint8_t valid[kMaxPairs];            // whether its id names an expert (else no more is said)
};
static_assert(sizeof(FewTable) == kFewTableBytes, "workspace");

// ... made by one workgroup of WAVES wavefronts, with scratch in LDS.
template <int WAVES>
__device__ void make_table(const Ids& ids, FewTable* out, uint32_t* bits, uint8_t (*lists)[kMaxPairs],
                           FewTable& tb) {
  const int lane = threadIdx.x & (kWave - 1), wv = threadIdx.x / kWave;
  mark_experts(ids, bits);
  if (wv == 0) {
    uint32_t m = lane < 32 ? bits[lane] : 0u;
    const int c = __popc(m), inc = scan32(c, lane);
    for (int at = inc - c; m; m &= m - 1)
      tb.active[at++] = static_cast<uint16_t>(lane * 32 + __ffs(m) - 1);
    if (lane == 31) tb.n = inc;
#pragma unroll
    for (int i = 0; i < kIds; ++i) tb.valid[lane + i * kWave] = ids.id[i] >= 0;
  }
  __syncthreads();
  for (int g = wv; g < tb.n; g += WAVES) {
    const int n = pairs_of(ids, tb.active[g], lane, lists[wv]);
    if (lane == 0) tb.start[g] = static_cast<uint16_t>(n);
  }
  __syncthreads();
  if (wv == 0) {
    int v[kIds], sum = 0, most = 0;
#pragma unroll
    for (int i = 0; i < kIds; ++i) {
      const int g = lane * kIds + i;
      v[i] = g < tb.n ? tb.start[g] : 0;
      sum += v[i];
      most = max(most, v[i]);
    }
    int at = sum;
    for (int off = 1; off < kWave; off <<= 1) {
      const int u = __shfl_up(at, off, kWave);
      if (lane >= off) at += u;
      most = max(most, __shfl_xor(most, off, kWave));
    }
    const int end = at;
    at -= sum;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < kIds; ++i) {
      if (lane * kIds + i <= tb.n) tb.start[lane * kIds + i] = static_cast<uint16_t>(at);
      at += v[i];
    }
    if (lane == kWave - 1) {
      tb.start[kMaxPairs] = static_cast<uint16_t>(end);  // where all 256 are groups
      tb.most = most;
    }
  }
  __syncthreads();
  for (int g = wv; g < tb.n; g += WAVES) {
    const int n = pairs_of(ids, tb.active[g], lane, lists[wv]), at = tb.start[g];
    for (int i = lane; i < n; i += kWave) {
      const int s = lists[wv][i];
      tb.pair[at + i] = static_cast<uint8_t>(s);
      tb.group[s] = static_cast<uint8_t>(g);
      tb.rank[s] = static_cast<uint8_t>(i);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < static_cast<int>(sizeof(FewTable) / 16); i += WAVES * kWave)
    reinterpret_cast<u32x4_t*>(out)[i] = reinterpret_cast<const u32x4_t*>(&tb)[i];
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

// 16 bytes at a uniform address and a lane's offset.
__device__ __forceinline__ u32x4_t load16(const uint8_t* base, uint32_t off) {
  return *reinterpret_cast<const u32x4_t*>(base + off);
}

__device__ __forceinline__ f32x4_t mma(bf16x8_t w, u32x4_t x, f32x4_t acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8_t, x), acc, 0, 0, 0);
}

// One wavefront's loads of weights: step s of its fragments.
template <int FR>
struct Weights {
  const uint8_t* p[FR];  // the fragments' first rows
  const float* scales[FR];  // e4m3: of the fragments' block rows
};
template <int KIND, int FR>
struct Loaded {
  u32x4_t w[FR];
  // `last`: the step whose second half lies past the contraction's end; there the
  // lanes of that half (`tail`) read the first
  __device__ __forceinline__ void load(const Weights<FR>& at, uint32_t off, int s, int last, int tail) {
    if (KIND != kFewBf16 && s == last) off -= tail * 64;
#pragma unroll
    for (int f = 0; f < FR; ++f) w[f] = load16(at.p[f] + static_cast<int64_t>(s) * 128, off);
  }
};

// Steps [from, to) of a contraction of K, into acc.  `first` holds step `from`
// already and is left with step next_from of `next`: the loads of what comes next
// are under way while a step is worked on, the tokens' ahead of them, since loads
// come back in the order of their issue.
//  off  this lane's place in a fragment's load
//  x    the tokens (NB of them a lane, at xo), or the PARTS of h, `apart` bytes from
//       one another.  Lanes without a token read another one's: no one reads their
//       sums.
template <int KIND, int FR, int NB, int PARTS>
__device__ __forceinline__ void steps(const Weights<FR>& at, uint32_t off, Loaded<KIND, FR>& first,
                                      int from, int to, int K, const Weights<FR>& next, int next_from,
                                      const uint8_t* x, const uint32_t (&xo)[NB], int64_t apart,
                                      int tail, f32x4_t (&acc)[FR][NB]) {
  using F = Fmt<KIND>;
  constexpr int kPer = KIND == kFewBf16 ? 1 : 2;  // matrix instructions per load and token
  const int last = K % F::kStep ? K / F::kStep : -1;
  u32x4_t v[kPer][NB][PARTS];
  auto tokens = [&](int s) {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
          uint32_t o = xo[b] + i * 16;
          if (KIND != kFewBf16 && s == last) o -= tail * (F::kHalf * 2);
          v[i][b][p] = load16(x + p * apart + static_cast<int64_t>(s) * (F::kStep * 2), o);
        }
  };
  auto work = [&](const Loaded<KIND, FR>& l, int s) {
    if (KIND != kFewBf16 && s == last) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int p = 0; p < PARTS; ++p)
            if (tail) v[i][b][p] = u32x4_t{0, 0, 0, 0};
    }
#pragma unroll
    for (int f = 0; f < FR; ++f) {
      f32x4_t sum[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) sum[b] = KIND == kFewE4m3 ? f32x4_t{0, 0, 0, 0} : acc[f][b];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        bf16x8_t c;
        if constexpr (KIND == kFewBf16)
          c = __builtin_bit_cast(bf16x8_t, l.w[f]);
        else
          c = widen<KIND>(l.w[f][2 * i], l.w[f][2 * i + 1]);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int p = 0; p < PARTS; ++p) sum[b] = mma(c, v[i][b][p], sum[b]);
      }
      static_assert(KIND != kFewE4m3 || F::kStep == kBlock, "a load is a block of scales");
      const float scale = KIND == kFewE4m3 ? at.scales[f][s] : 1.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[f][b][j] = KIND == kFewE4m3 ? fmaf(scale, sum[b][j], acc[f][b][j]) : sum[b][j];
    }
  };
  Loaded<KIND, FR> second;
  for (int s = from; s < to; s += 2) {
    const bool two = s + 1 < to, more = s + 2 < to;
    tokens(s);
    second.load(at, off, min(s + 1, to - 1), last, tail);
    __builtin_amdgcn_sched_barrier(0);
    work(first, s);
    __builtin_amdgcn_sched_barrier(0);
    if (two) tokens(s + 1);
    first.load(more ? at : next, off, more ? s + 2 : next_from, last, tail);
    __builtin_amdgcn_sched_barrier(0);
    if (two) work(second, s + 1);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// The sum of a fragment's two parts for column ln.chunk() of token ln.row: a lane's
// results are columns 2 q and 2 q + 1 of its own part, then of none; its neighbour
// has the other part of both.
__device__ __forceinline__ float both_parts(f32x4_t v, const Lane& ln) {
  const float keep = ln.part ? v[3] : v[0], give = ln.part ? v[1] : v[2];
  return keep + __uint_as_float(dpp_u32<0xB1>(__float_as_uint(give)));  // the neighbour's
}

// ---------------------------------------------------------------------------
// gate and up: a workgroup takes 8 columns of one expert's h: each wavefront the
// gate's and the up's rows over a quarter of the contraction.
// ---------------------------------------------------------------------------
constexpr int kGuFrags = 2;  // the gate's and the up's
constexpr int kGuWaves = 4, kGuThreads = kGuWaves * kWave;

// MANY: up to 16 tokens in one pass over an expert's weights, else 8.
template <int KIND, int PARTS, bool MANY>
__global__ __launch_bounds__(kGuThreads) void few_gate_up(FewLayer g, int tiles) {
  using F = Fmt<KIND>;
  constexpr int kPassRows = MANY ? 16 : 8;
  __shared__ float part[kGuWaves][kGuFrags][kPassRows][kCols + 1];
  __shared__ uint32_t bits[kMaxIds / 32];
  __shared__ uint8_t lists[kGuWaves][kMaxPairs];
  const int t = threadIdx.x, lane = t & (kWave - 1);
  const int wv = __builtin_amdgcn_readfirstlane(t / kWave);
  if (blockIdx.x == 0) {  // one more workgroup: the grouping for the other kernel
    __shared__ FewTable tb;
    make_table<kGuWaves>(load_ids(g, lane), static_cast<FewTable*>(g.table), bits, lists, tb);
    return;
  }
  const int id = static_cast<int>(blockIdx.x) - 1, n0 = id % tiles * kCols;
  int slot = id / tiles;
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
  const Lane ln(lane);
  const uint8_t* wbase = static_cast<const uint8_t*>(shared ? g.shared_gate_up : g.gate_up);
  const float* sbase = shared ? g.shared_gate_up_scales : g.gate_up_scales;
  Weights<kGuFrags> at;
#pragma unroll
  for (int f = 0; f < kGuFrags; ++f) {
    const int row = f * g.f + n0;  // the gate's, the up's
    at.p[f] = wbase + (static_cast<int64_t>(e) * 2 * g.f + row) * g.d * F::kElem;
    at.scales[f] = KIND != kFewE4m3 ? nullptr
                                    : sbase + (static_cast<int64_t>(e) * ((2 * g.f + kBlock - 1) / kBlock) +
                                               row / kBlock) * ((g.d + kBlock - 1) / kBlock);
  }
  const uint32_t off = static_cast<uint32_t>(ln.row * g.d * F::kElem + ln.chunk() * 16);
  const int all = (g.d + F::kStep - 1) / F::kStep;
  const int from = all * wv / kGuWaves, to = all * (wv + 1) / kGuWaves;
  const int last = g.d % F::kStep ? g.d / F::kStep : -1;
  Loaded<KIND, kGuFrags> w;
  w.load(at, off, min(from, all - 1), last, ln.tail);
  for (int m0 = 0; m0 < n; m0 += kPassRows) {
    auto pass = [&](auto nb) {
      constexpr int NB = decltype(nb)::value;
      f32x4_t acc[kGuFrags][NB];
      uint32_t xo[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int r = min(m0 + b * 8 + ln.row, n - 1);
        const int token = shared ? r : list[r] / g.k;
        xo[b] = static_cast<uint32_t>(token * g.d + ln.chunk() * F::kChunk) * 2;
        acc[0][b] = acc[1][b] = f32x4_t{0, 0, 0, 0};
      }
      steps<KIND, kGuFrags, NB, 1>(at, off, w, from, to, g.d, at, min(from, all - 1),
                         static_cast<const uint8_t*>(g.x), xo, 0, ln.tail, acc);
#pragma unroll
      for (int f = 0; f < kGuFrags; ++f)
#pragma unroll
        for (int b = 0; b < NB; ++b)
          part[wv][f][b * 8 + ln.row][ln.chunk()] = both_parts(acc[f][b], ln);
    };
    if constexpr (MANY) {
      if (n - m0 > 8)
        pass(std::integral_constant<int, 2>{});
      else
        pass(std::integral_constant<int, 1>{});
    } else {
      pass(std::integral_constant<int, 1>{});
    }
    __syncthreads();
    const int r = t / kCols, c = t % kCols;
    if (r < kPassRows && m0 + r < n) {
      float gate = 0.0f, up = 0.0f;
#pragma unroll
      for (int w = 0; w < kGuWaves; ++w) {
        gate += part[w][0][r][c];
        up += part[w][1][r][c];
      }
      if (KIND == kFewInt8) {
        const float* s = sbase + static_cast<int64_t>(e) * 2 * g.f + n0 + c;
        gate *= s[0];
        up *= s[g.f];
      }
      float h = silu(gate) * up;
      const int row = shared ? g.T * g.k + m0 + r : list[m0 + r];
      uint16_t* out = g.h + static_cast<int64_t>(row) * g.f + n0 + c;
#pragma unroll
      for (int p = 0; p < PARTS; ++p) {
        uint16_t v = f32_to_bf16(h);
        // what is finite but rounds to an infinity takes bf16's largest
        if ((v & 0x7FFFu) == 0x7F80u && fabsf(h) < __builtin_inff()) --v;
        out[p * g.h_apart] = v;
        h -= bf16_to_f32(v);
        if (h != h) h = 0.0f;  // what is not finite has no rest
      }
    }
    __syncthreads();
  }
}
static_assert(kGuThreads >= 16 * kCols, "a thread per element of h");

// ---------------------------------------------------------------------------
// down and combine: a workgroup takes 8 to 32 columns of out, FR fragments (down_plan).
// Its wavefronts share the
// steps of all the experts hit evenly, each a contiguous range of them; an
// expert's sums are left in LDS by the wavefront that begins it, those of a
// wavefront that begins inside one beside them, and one meeting later they are
// weighted and added up in the pairs' order.
// ---------------------------------------------------------------------------
constexpr int kDnWaves = 16, kDnThreads = kDnWaves * kWave;
constexpr int kEdgeRows = 32;  // rows of an expert that wavefronts may share

// Wavefront w's first step of `total`: a multiple of `grain`.
__device__ __forceinline__ int first_step(int w, int waves, int total, int grain) {
  return static_cast<int>(static_cast<int64_t>(w) * (total / grain) / waves) * grain;
}

template <int KIND, int PARTS, bool MANY, int FR>
__global__ __launch_bounds__(kDnThreads) void few_down(FewLayer g, int splits) {
  using F = Fmt<KIND>;
  constexpr int kDnCols = FR * kCols, kDnPitch = kDnCols + 4;
  constexpr int kPassRows = MANY ? 16 : 8;
  // sums by pair, then by token (the shared expert's)
  __shared__ __align__(16) float sums[kMaxPairs + kFewTokens][kDnPitch];
  __shared__ __align__(16) float edge[kDnWaves][kEdgeRows][kDnPitch];
  __shared__ FewTable tb;
  __shared__ float weight[kMaxPairs];
  __shared__ int inside[kDnWaves];  // which of the experts a wavefront begins inside of, or -1
  const int t = threadIdx.x, lane = t & (kWave - 1);
  const int wv = __builtin_amdgcn_readfirstlane(t / kWave);
  const int n0 = static_cast<int>(blockIdx.x) * kDnCols;
  const int pairs = g.T * g.k;
  const FewTable* table = static_cast<const FewTable*>(g.table);
  const int groups = __builtin_amdgcn_readfirstlane(table->n) + g.shared;
  const int all = (g.f + F::kStep - 1) / F::kStep, total = groups * all;
  // an expert with more rows than `edge` holds is one wavefront's
  const int grain = __builtin_amdgcn_readfirstlane(table->most) > kEdgeRows ? all : 1;
  const int split = blockIdx.y, waves = splits * kDnWaves;
  const int begin = first_step(split * kDnWaves + wv, waves, total, grain);
  const int end = first_step(split * kDnWaves + wv + 1, waves, total, grain);
  // this workgroup's steps: it holds the sums of the experts that begin here
  const int wg_begin = first_step(split * kDnWaves, waves, total, grain);
  const int wg_end = first_step((split + 1) * kDnWaves, waves, total, grain);

  const Lane ln(lane);
  const uint32_t off = static_cast<uint32_t>(ln.row * g.f * F::kElem + ln.chunk() * 16);
  const int last = g.f % F::kStep ? g.f / F::kStep : -1;
  auto weights_of = [&](int grp, int e) {
    const bool shared = grp < g.shared;
    const uint8_t* wbase = static_cast<const uint8_t*>(shared ? g.shared_down : g.down);
    const float* sbase = shared ? g.shared_down_scales : g.down_scales;
    Weights<FR> r;
#pragma unroll
    for (int f = 0; f < FR; ++f) {
      const int col = min(n0 + f * kCols, g.d - kCols);  // fragments past out repeat the last
      r.p[f] = wbase + (static_cast<int64_t>(e) * g.d + col) * g.f * F::kElem;
      r.scales[f] = KIND != kFewE4m3
                        ? nullptr
                        : sbase + (static_cast<int64_t>(e) * ((g.d + kBlock - 1) / kBlock) +
                                   col / kBlock) * ((g.f + kBlock - 1) / kBlock);
    }
    return r;
  };
  Loaded<KIND, FR> w;
  Weights<FR> at;
  int grp = begin / all, e = 0;
  if (begin < end) {  // the first weights, ahead of the rest of the table
    if (grp >= g.shared) e = __builtin_amdgcn_readfirstlane(table->active[grp - g.shared]);
    at = weights_of(grp, e);
    w.load(at, off, begin - grp * all, last, ln.tail);
  }
  for (int i = t; i < static_cast<int>(sizeof(FewTable) / 16); i += kDnThreads)
    reinterpret_cast<u32x4_t*>(&tb)[i] = reinterpret_cast<const u32x4_t*>(table)[i];
  if (t < pairs) weight[t] = g.topk_w[t];
  if (lane == 0) inside[wv] = begin < end && begin > grp * all ? grp : -1;
  __syncthreads();

  for (int s = begin; s < end; ++grp) {
    const int from = s - grp * all, to = min(all, from + end - s);
    s += to - from;
    const bool shared = grp < g.shared;
    const int first = shared ? 0 : tb.start[grp - g.shared];
    const int n = __builtin_amdgcn_readfirstlane(shared ? g.T : tb.start[grp - g.shared + 1] - first);
    int next_e = e;
    Weights<FR> next = at;
    if (s < end) {
      next_e = __builtin_amdgcn_readfirstlane(tb.active[grp + 1 - g.shared]);
      next = weights_of(grp + 1, next_e);
    }
    const float* sbase = shared ? g.shared_down_scales : g.down_scales;
    for (int m0 = 0; m0 < n; m0 += kPassRows) {
      const bool again = m0 + kPassRows < n;  // these weights with other rows
      auto pass = [&](auto nb) {
        constexpr int NB = decltype(nb)::value;
        f32x4_t acc[FR][NB];
        int row[NB];
        uint32_t xo[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const int r = min(m0 + b * 8 + ln.row, n - 1);
          row[b] = shared ? pairs + r : tb.pair[first + r];
          xo[b] = static_cast<uint32_t>(row[b] * g.f + ln.chunk() * F::kChunk) * 2;
#pragma unroll
          for (int f = 0; f < FR; ++f) acc[f][b] = f32x4_t{0, 0, 0, 0};
        }
        steps<KIND, FR, NB, PARTS>(at, off, w, from, to, g.f, again ? at : next,
                               again ? from : s < end ? 0 : from,
                               reinterpret_cast<const uint8_t*>(g.h), xo, g.h_apart * 2, ln.tail, acc);
#pragma unroll
        for (int f = 0; f < FR; ++f) {
          float sc = 1.0f;
          if constexpr (KIND == kFewInt8)
            sc = sbase[static_cast<int64_t>(e) * g.d + min(n0 + f * kCols, g.d - kCols) + ln.chunk()];
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const float v = both_parts(acc[f][b], ln) * sc;
            const int r = m0 + b * 8 + ln.row;
            if (r < n) (from == 0 ? sums[row[b]] : edge[wv][r])[f * kCols + ln.chunk()] = v;
          }
        }
      };
      if constexpr (MANY) {
        if (n - m0 > 8)
          pass(std::integral_constant<int, 2>{});
        else
          pass(std::integral_constant<int, 1>{});
      } else {
        pass(std::integral_constant<int, 1>{});
      }
    }
    at = next;
    e = next_e;
  }
  __syncthreads();
  // what wavefronts that began inside an expert hold of it
  for (int o = t; o < (pairs + (g.shared ? g.T : 0)) * kDnCols; o += kDnThreads) {
    const int row = o / kDnCols, c = o % kDnCols;
    if (row < pairs && !tb.valid[row]) continue;
    const int grp = row < pairs ? tb.group[row] + g.shared : 0;
    const int rank = row < pairs ? tb.rank[row] : row - pairs;
    float y = grp * all >= wg_begin && grp * all < wg_end ? sums[row][c] : 0.0f;
#pragma unroll
    for (int w = 0; w < kDnWaves; ++w)
      if (inside[w] == grp) y += edge[w][rank][c];
    sums[row][c] = y;
  }
  __syncthreads();
  for (int o = t; o < g.T * kDnCols; o += kDnThreads) {
    const int tok = o / kDnCols, c = o % kDnCols;
    if (n0 + c >= g.d) continue;
    float v = 0.0f;
#pragma unroll 4
    for (int j = 0; j < g.k; ++j) {
      const int s = tok * g.k + j;
      // an expert without steps here has no part in this sum, whatever its weight
      const int at = (tb.group[s] + g.shared) * all;
      if (tb.valid[s] && at < wg_end && at + all > wg_begin) v = fmaf(weight[s], sums[s][c], v);
    }
    if (g.shared) v += sums[pairs + tok][c];
    const int64_t at = static_cast<int64_t>(tok) * g.d + n0 + c;
    if (splits > 1)
      g.parts[split * g.T * g.d + at] = v;
    else if (g.out_f32)
      static_cast<float*>(g.out)[at] = v;
    else
      static_cast<uint16_t*>(g.out)[at] = f32_to_bf16(v);
  }
}
static_assert(kMaxPairs <= kDnThreads, "a thread per pair");

// out = the splits' sum, in their order.
__global__ __launch_bounds__(256) void few_join(FewLayer g, int splits) {
  const int n = g.T * g.d, i = static_cast<int>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n) return;
  float v = g.parts[i];
#pragma unroll 4
  for (int z = 1; z < splits; ++z) v += g.parts[z * n + i];
  if (g.out_f32)
    static_cast<float*>(g.out)[i] = v;
  else
    static_cast<uint16_t*>(g.out)[i] = f32_to_bf16(v);
}

// How few_down is laid out: the fragments of a wavefront (8 columns of out each)
// and the workgroups that share the steps of one tile of out.
struct DownPlan {
  int frags, splits;
};

// A workgroup for each CU, or as many of them as go: us of the layer with 1, 2, 3, 4
// fragments, 1 token on bf16, 8 on integers and 32 on bf16 over 64 experts of f = 1024
// (2048 where d = 6144):
//   d = 2048  25.7  26.8  27.7  27.8 and  70  67  70  68 and 168 160 170 155
//   d = 2560  37.5  31.8  32.2  32.8      98  82  77  77     248 218 197 190
//   d = 4096  48.3  43.6  45.0  46.2     122 107 114 110     321 291 310 284
//   d = 6144   119   117   110   111     320 304 276 284     930 929 845 857
// Short calls (fewer than kLongSteps steps of all experts) take the fewest
// fragments that suffice.  In longer ones what is read of h counts beside the
// weights, two fragments share it, and a third kernel that joins the sums of
// workgroups that split the steps (3 us and a launch) costs less than CUs without
// work: of the layouts that use most CUs, the one with two fragments or the
// fewest more, or the most for many tokens on bf16 with 16 steps an expert (8 steps,
// 32 tokens over 128 of 1024 x 512 76.8 us with two, 80.0 with four; 12 tokens over 64
// of 2048 x 1024 121 and 123, 20 over 16 of 4096 x 4096 353 and 323; codes, which need more
// registers, 32 over 64 of 2048 x 1024 110 and 123).  Steps are split where that
// leaves a wavefront kSplitSteps steps if every pair has an expert of its own, in
// short calls too.  us without, with 4 and with 2: 28 tokens over 5 experts of
// 128 x 3584 104, 48, 38; 26 over 31 of 256 x 640 34 (4 does not split them), 29; 2
// over 59 of 320 x 704 16 (likewise), 18.
//
// On codes with more than 8 tokens the wider layouts do not fit a workgroup's 128
// registers: bytes of scratch a lane with 3 and 4 fragments 56 and 132 (e4m3, out of
// f32), 0 and 80 (e4m3, bf16), 12 and 88 (integers, f32), 0 and 12 (integers, bf16).  d
// above 6144 takes 4, d = 6144 3, long calls on narrower layers 2 to 4.
constexpr int kMaxSplits = 16, kSplitSteps = 2, kLongSteps = 256, kMaxFrags = 4;
DownPlan down_plan(int T, int k, int d, int f, int E, bool shared, int step) {
  const int pairs = T * k, cols = d / kCols;
  const int64_t steps =
      static_cast<int64_t>((pairs < E ? pairs : E) + shared) * ((f + step - 1) / step);
  auto splits_of = [&](int frags) {
    int64_t s = kCus / ((cols + frags - 1) / frags);
    const int64_t most = steps / (kDnWaves * kSplitSteps);
    if (s > most) s = most;
    if (s > kMaxSplits) s = kMaxSplits;
    return s > 1 ? static_cast<int>(s) : 1;
  };
  const int least = (cols + kCus - 1) / kCus;
  DownPlan best{least, splits_of(least)};
  if (steps < kLongSteps) return best;
  const bool most = step == Fmt<kFewBf16>::kStep && T > 16 && f / step >= 16;
  auto used = [&](const DownPlan& p) { return (cols + p.frags - 1) / p.frags * p.splits; };
  for (int frags = least + 1; frags <= kMaxFrags; ++frags) {
    const DownPlan p{frags, splits_of(frags)};
    if (used(p) > used(best) || (used(p) == used(best) && (most || best.frags == 1))) best = p;
  }
  return best;
}

template <int KIND, int PARTS, bool MANY>
hipError_t go(const FewLayer& g, hipStream_t stream) {
  const int pairs = g.T * g.k, tiles = g.f / kCols;
  const int slots = (pairs < g.E ? pairs : g.E) + g.shared;
  const hipError_t e = launch(few_gate_up<KIND, PARTS, MANY>, dim3(static_cast<uint32_t>(slots * tiles + 1)),
                              dim3(kGuThreads), 0, stream, g, tiles);
  if (e != hipSuccess) return e;
  const DownPlan plan = down_plan(g.T, g.k, g.d, g.f, g.E, g.shared, Fmt<KIND>::kStep);
  auto down = [&](auto fr) {
    constexpr int FR = decltype(fr)::value;
    return launch(few_down<KIND, PARTS, MANY, FR>,
                  dim3(static_cast<uint32_t>((g.d / kCols + FR - 1) / FR), plan.splits),
                  dim3(kDnThreads), 0, stream, g, plan.splits);
  };
  hipError_t err;
  switch (plan.frags) {
    case 1: err = down(std::integral_constant<int, 1>{}); break;
    case 2: err = down(std::integral_constant<int, 2>{}); break;
    case 3: err = down(std::integral_constant<int, 3>{}); break;
    default: err = down(std::integral_constant<int, 4>{});
  }
  if (plan.splits == 1 || err != hipSuccess) return err;
  return launch(few_join, dim3(static_cast<uint32_t>((g.T * g.d + 255) / 256)), dim3(256), 0, stream,
                g, plan.splits);
}
template <int KIND>
hipError_t go(const FewLayer& g, hipStream_t stream) {
  if (g.T > 8) return g.out_f32 ? go<KIND, 3, true>(g, stream) : go<KIND, 2, true>(g, stream);
  return g.out_f32 ? go<KIND, 3, false>(g, stream) : go<KIND, 2, false>(g, stream);
}

}  // namespace

// The grouping, h, and the splits' sums, whatever the weights are held in.
FewScratch few_scratch(int T, int k, int d, int f, int E, bool shared) {
  FewScratch s;
  s.h = kFewTableBytes;
  const size_t h = static_cast<size_t>(T) * (k + shared) * f * 3 * sizeof(uint16_t);
  s.parts = (s.h + h + 15) / 16 * 16;
  int splits = 1;
  for (int step : {Fmt<kFewBf16>::kStep, Fmt<kFewE4m3>::kStep, Fmt<kFewInt8>::kStep}) {
    const int n = down_plan(T, k, d, f, E, shared, step).splits;
    if (n > splits) splits = n;
  }
  s.bytes = s.parts + (splits > 1 ? static_cast<size_t>(splits) * T * d * sizeof(float) : 0);
  return s;
}

hipError_t launch_layer_few(const FewLayer& g, FewKind kind, hipStream_t stream) {
  switch (kind) {
    case kFewBf16: return go<kFewBf16>(g, stream);
    case kFewE4m3: return go<kFewE4m3>(g, stream);
    default: return go<kFewInt8>(g, stream);
  }
}

}  // namespace moe
