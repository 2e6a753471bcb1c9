// Matrix products over rows grouped by expert, on the bf16 matrix cores:
//   rows     y[p]  = W_e x[row(p)]                 p in [offsets[e], offsets[e+1])
//   input    dx[p] = W_e^T dy[p]
//   weights  dW_e  = sum over the group's p of dy[p] x[row(p)]^T
// and the first of them over e4m3 codes with a float32 scale per 128 columns
// of a row and per 128 x 128 weights, and over 8-bit integers with a float32
// scale per row of x and per row of W_e.
//
// All five are one loop: D[m][n] = sum_k R[m][k] F[n][k] over a tile of one
// group (256 x 256 where it has the rows), R being the operand whose index is
// the output's row and F the one whose index is its column.  A stage of the
// loop is 64 or 128 bytes of the contraction of every row of R and F in LDS,
// fetched by global_load_lds.  An operand that is contiguous along the
// contraction is stored [row][stage]; one that is contiguous along its own
// index (W of `input`, both operands of `weights`) is stored [stage][its
// columns] and read with the transposing ds_read_b64_tr_b16, so no operand is
// ever transposed in memory.
// Chunks past an operand's end are fetched from a zero block, so no tail of
// K, N or a group's rows needs a branch in the arithmetic, and both operands
// are zero there (no 0 * inf).  F goes to the matrix instruction's A side:
// a lane then holds four consecutive columns of one output row.
//
// What bounds it (measured): with few rows a group, the weights' bytes (8 rows
// over 8 of 256 experts, 403 MB: 75 us, 5.4 TB/s; the skewed 2048-token prompt,
// 13.0 GB: 2.45 ms, 5.3 TB/s).  With many, LDS: a 32-deep stage of a 256 x 256
// tile takes 1024 cycles of the matrix cores and as many of LDS (96 KB of
// fragment reads, 32 KB of fetches at 128 bytes a cycle), one half's reads
// against the other's products; 8192 rows over one 4096 x 4096 matrix run at
// 1150-1190 TFLOP/s in all, over 8192 x 8192 at 1310.  Codes run their products
// at the same rate with the widening beside them: 930 TFLOP/s (297 us) there.
// Integers have half the bytes and twice the rate, so the same balance: 8192
// rows over 4096 x 4096 118 us, over 8192 x 8192 427 us (2.33 and 2.58 POP/s), 64
// groups of 512 rows over 2048 x 2048 166 us (1.66), where each tile's 32 stages
// hardly hide its start and its stores; 64 rows over 57 of 256 experts of 4096 x 6144
// 225 us (6.4 TB/s), the skewed 2048-token prompt 1.24 ms (5.3 TB/s).
#include <type_traits>

#include "common.h"
#include "launch.h"
#include "lds_dma.h"

namespace moe {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
// read by scalar loads: a vector load's wait would drain the fetches into LDS
typedef const __attribute__((address_space(4))) int32_t const_i32;
typedef const __attribute__((address_space(4))) float const_f32;

constexpr int kBlock = 128;       // columns (and weight rows) per scale

// What a fetch past an operand's end reads.
__device__ const uint4 g_zero[8] = {};

// kWeightsBy: kWeights with x gathered through rows.
enum Kind { kRows, kInput, kWeights, kWeightsBy, kCodes, kInts };

// This wavefront's fetches but the newest N done and its LDS reads back, then
// every wavefront of the workgroup here.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"i"(N) : "memory");
}

// This wavefront's LDS reads back, then a meeting; nothing is scheduled across.
__device__ __forceinline__ void reads_and_meet() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
template <int N>
__device__ __forceinline__ void wait_fetches() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"i"(N) : "memory");
}

__device__ __forceinline__ const uint8_t* zero_block() {
  return reinterpret_cast<const uint8_t*>(g_zero);
}

// n / div for 0 <= n < 2^24 and div <= 256; magic = ceil(2^32 / div), 0 for 1.
__device__ __forceinline__ uint32_t row_div(uint32_t n, uint32_t magic) {
  return magic ? __umulhi(n, magic) : n;
}

// Eight e4m3 codes as bf16, exactly.
__device__ __forceinline__ bf16x8_t codes_to_bf16(uint32_t lo, uint32_t hi) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return f32_to_bf16(lo) | (static_cast<uint32_t>(f32_to_bf16(hi)) << 16);
}

// The product of two fragments of 16 rows x 128 codes (two 16-byte chunks a
// lane, in the same places of both), as bf16: exact products, float32 sums.
// The 8-bit matrix instructions have twice the rate, but align the products of
// neighbouring codes to the largest before they add them: where a block's large
// products cancel, what is left came out 5% off (448 * 448 - 448 * 448 beside
// products of integers up to 15), more than a bf16 result's own rounding.
__device__ __forceinline__ f32x4_t codes_product(const u32x4_t (&f)[2], const u32x4_t (&r)[2]) {
  f32x4_t p{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int v = 0; v < 4; v += 2)
      p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_to_bf16(f[h][v], f[h][v + 1]),
                                                  codes_to_bf16(r[h][v], r[h][v + 1]), p, 0, 0, 0);
  return p;
}

// One matrix instruction over 64 bytes of the contraction: 32 bf16 values, or
// 64 integers, whose int32 sums are exact (K <= 65536 products of at most 2^14).
__device__ __forceinline__ f32x4_t mma(u32x4_t f, u32x4_t r, f32x4_t acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, f),
                                                 __builtin_bit_cast(bf16x8_t, r), acc, 0, 0, 0);
}
__device__ __forceinline__ i32x4_t mma(u32x4_t f, u32x4_t r, i32x4_t acc) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, f),
                                               __builtin_bit_cast(i32x4_t, r), acc, 0, 0, 0);
}

struct Group {
  int e, a, b;  // expert, its grouped positions
  int t;        // this workgroup's row tile of the group
  int n;        // the group's row tiles that come together with it
  int high;     // how many of them, the first ones, are kExtraRows higher
};

// The group's bounds as the kernels take them: whatever offsets holds, they
// lie in [0, P].
__device__ __forceinline__ void group_bounds(const GroupedMm& g, int e, int& a, int& b) {
  a = min(max(g.offsets[e], 0), g.P);
  b = min(max(g.offsets[e + 1], a), g.P);
}

// Which group holds row tile `tile`: every thread takes a few groups, a scan
// over the workgroup gives their first tiles, and the owner tells the others.
// e = -1 past the last tile.  Groups have ceil(rows / BM) tiles, in ascending
// order of the groups; with `tall_first`, the tiles of more than BM / 2 rows
// come before all others.  EXTRA: the last tile's rows are spread over the
// others, EXTRA each, where they suffice.
template <int BM, int THREADS, int EXTRA = 0>
__device__ Group find_group(const GroupedMm& g, int64_t tile, bool tall_first, int* sh) {
  constexpr int kPer = 1024 / THREADS, kWaves = THREADS / kWave;  // E <= 1024
  const int t = threadIdx.x, lane = t & (kWave - 1), wv = t / kWave;
  int a[kPer], b[kPer], n[kPer], low[kPer], high[kPer], inc = 0, inc_low = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    a[i] = b[i] = high[i] = 0;
    if (kPer * t + i < g.E) group_bounds(g, kPer * t + i, a[i], b[i]);
    n[i] = (b[i] - a[i] + BM - 1) / BM;
    int rest = (b[i] - a[i]) % BM;
    if (EXTRA > 0 && rest > 0 && rest <= EXTRA * (n[i] - 1)) {
      high[i] = (rest + EXTRA - 1) / (EXTRA > 0 ? EXTRA : 1);
      rest = 0;
      --n[i];
    }
    low[i] = tall_first && rest > 0 && rest <= BM / 2;  // its last tile goes to the end
    n[i] -= low[i];
    inc += n[i];
    inc_low += low[i];
  }
  const int mine = inc, mine_low = inc_low;
  for (int off = 1; off < kWave; off <<= 1) {
    const int v = __shfl_up(inc, off, kWave), u = __shfl_up(inc_low, off, kWave);
    if (lane >= off) {
      inc += v;
      inc_low += u;
    }
  }
  if (t == 0) sh[2 * kWaves] = -1;
  if (lane == kWave - 1) {
    sh[wv] = inc;
    sh[kWaves + wv] = inc_low;
  }
  __syncthreads();
  int first = inc - mine, first_low = inc_low - mine_low;
  for (int w = 0; w < kWaves; ++w) {
    if (w < wv) {
      first += sh[w];
      first_low += sh[kWaves + w];
    }
    first_low += sh[w];  // behind all the others
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const bool mid = tile >= first && tile < first + n[i], end = low[i] && tile == first_low;
    if (mid || end) {
      sh[2 * kWaves] = kPer * t + i;
      sh[2 * kWaves + 1] = a[i];
      sh[2 * kWaves + 2] = b[i];
      sh[2 * kWaves + 3] = mid ? static_cast<int>(tile) - first : n[i];
      sh[2 * kWaves + 4] = mid ? n[i] : 0;
      sh[2 * kWaves + 5] = high[i];
    }
    first += n[i];
    first_low += low[i];
  }
  __syncthreads();
  Group r{sh[2 * kWaves], sh[2 * kWaves + 1], sh[2 * kWaves + 2], sh[2 * kWaves + 3],
          sh[2 * kWaves + 4], sh[2 * kWaves + 5]};
  __syncthreads();
  return r;
}

// Row of x (or of the codes) at grouped position p; -1 where it has none.
__device__ __forceinline__ int64_t source_row(const GroupedMm& g, int p) {
  if (!g.rows) return p;
  const uint32_t s = static_cast<uint32_t>(g.rows[p]);
  return s < g.row_limit ? static_cast<int64_t>(row_div(s, g.div_magic)) : -1;
}

// WM x WN wavefronts, each with RF x FF fragments of 16 x 16 outputs.
template <int KIND, int WM_, int WN_, int RF_, int FF_, int NST_, int SB_ = 128, bool PP_ = false>
struct Cfg {
  static constexpr int K = KIND, WM = WM_, WN = WN_, RF = RF_, FF = FF_, NST = NST_;
  static constexpr bool PP = PP_;      // the two halves of the workgroup in turn
  static constexpr int SB = SB_;       // bytes of the contraction per stage and row
  static constexpr int SR = SB / 2;    // the same as bf16 elements
  static constexpr int KK = SB / 64;   // matrix instructions' halves of a stage
  static constexpr int CPR = SB / 16;  // 16-byte chunks of it
  static constexpr int Waves = WM * WN, Threads = Waves * kWave;
  static constexpr int BM = WM * RF * 16, BN = WN * FF * 16;
  static constexpr bool DW = KIND == kWeights || KIND == kWeightsBy;
  static constexpr bool RT = DW;                    // R contiguous along m
  static constexpr bool FT = DW || KIND == kInput;  // F contiguous along n
  static constexpr bool F8 = KIND == kCodes, I8 = KIND == kInts;
  using Acc = std::conditional_t<I8, i32x4_t, f32x4_t>;
  static constexpr int RBytes = BM * SB, FBytes = BN * SB;
  static constexpr int SBytes = F8 ? Threads * 4 : 0;  // a stage's row scales
  static constexpr int Stage = RBytes + FBytes + SBytes;
  static constexpr int Lds = Stage * NST;
  // fetches per wavefront and stage; R's wrap around where they do not divide
  static constexpr int RI = (RBytes + Waves * 1024 - 1) / (Waves * 1024);
  static constexpr int FI = FBytes / (Waves * 1024);
  static constexpr int Fetches = RI + FI + (F8 ? 1 : 0);
  static_assert(Lds <= 160 * 1024, "LDS");
};

// Swizzle of the [row][stage] layout with 128-byte stages: chunk c of row r is stored at
// c ^ ((r >> 1) & 7), so the 16 rows a fragment read touches at once lie in
// different banks.  The DMA writes LDS in lane order; the lanes pick their
// sources accordingly.
// With 64-byte rows four rows share the banks: c ^ (-(r >> 2) & 3).  A 16-byte
// read goes through lanes 0-3, 12-15 and 20-27 together (and so on): rows 0-3
// and 12-15 of one chunk with rows 4-11 of the next, which c ^ ((r >> 2) & 3)
// puts into the same banks (24-37% of LDS's cycles; 8192 rows over 4096 x 4096
// 234 us against 230, 64 groups of 512 rows over 2048 x 2048 347 against 338).
template <int SB>
__device__ __forceinline__ int kc_slot(int row, int chunk) {
  return SB == 128 ? chunk ^ ((row >> 1) & 7) : chunk ^ (-(row >> 2) & 3);
}
// ... of the [stage][columns] layout: 32-byte segment s of row r is stored at
// s ^ f(r), f from the three bits in which the eight rows that a transposing
// read of half a wavefront touches differ.
__device__ __forceinline__ int mn_swz(int row) { return (row & 3) | (((row >> 3) & 1) << 2); }

// This lane's fetches of one operand: at stage s its chunk j comes from
// p[j] + s * step where s * unit + off[j] < limit (the chunk lies before the
// contraction's end), else from the zero block.  unit: contraction bytes of a
// stage (operand contiguous along the contraction) or rows (the other kind).
constexpr int kNever = 1 << 30;  // off of a chunk that no stage has
template <int NI>
struct Src {
  const uint8_t* p[NI];
  int off[NI];
  int step;
};
template <int NI, int UNIT>
__device__ __forceinline__ void fetch(const Src<NI>& s, int stage, int limit, uint32_t lds,
                                      int first, int n_instr) {
#pragma unroll
  for (int j = 0; j < NI; ++j) {
    const uint8_t* p = s.p[j] + static_cast<int64_t>(stage) * s.step;
    dma16(stage * UNIT + s.off[j] < limit ? p : zero_block(),
          lds + ((first + j) % n_instr) * 1024);
  }
}

// One operand fragment: 16 rows x 64 contraction bytes (part `kk` of a
// stage), 16 bytes per lane.
template <int SB>
__device__ __forceinline__ u32x4_t frag_k(const uint8_t* st, int row0, int kk, int lane) {
  const int row = row0 + (lane & 15);
  return *reinterpret_cast<const u32x4_t*>(st + row * SB +
                                           (kc_slot<SB>(row, kk * 4 + (lane >> 4)) << 4));
}
// ... of the [stage][width] layout: 16 columns x 32 of the contraction.  Two
// transposing reads; in each, 16 lanes name four rows of 16 columns and get
// four rows of their own column.
template <int WIDTH>
__device__ __forceinline__ u32x4_t frag_mn(const uint8_t* st, int col0, int kk, int lane) {
  const int i = lane & 15, grp = lane >> 4;
  const int row = kk * 32 + grp * 8 + (i >> 2);
  const uint8_t* p = st + row * (WIDTH * 2) + (((col0 >> 4) ^ mn_swz(row)) << 5) + (i & 3) * 8;
  const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
  const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * WIDTH * 2));
  return __builtin_bit_cast(u32x4_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Output tile [m0, mend) x [n0, n0 + BN) of a group whose contraction is
// [0, red) (kWeights: positions [ga, gb)).
template <class C>
__device__ void tile(const GroupedMm& g, uint8_t* smem, int e, int m0, int mend, int n0, int ga,
                     int gb, void* out, bool out_f32) {
  const int t = threadIdx.x, lane = t & (kWave - 1);
  const int wv = __builtin_amdgcn_readfirstlane(t / kWave);
  const int wm = wv % C::WM, wn = wv / C::WM;
  const int elem = C::F8 || C::I8 ? 1 : 2;
  const int64_t wsz = static_cast<int64_t>(g.N) * g.K * elem;
  const int red = C::DW ? gb - ga : C::K == kInput ? g.N : g.K;
  const int red_bytes = C::RT ? 0 : red * elem;
  const int stages = C::RT ? (red + C::SR - 1) / C::SR : (red_bytes + C::SB - 1) / C::SB;
  const uint32_t lds0 = lds_addr(smem);

  // ---- sources
  constexpr int kUnitK = C::SB, kUnitMN = C::SR;
  Src<C::RI> rs;
  Src<C::FI> fs;
  const uint8_t* sp = zero_block();  // this lane's row scale
  int sstep = 0;
  // an operand contiguous along its own index, W columns from c0 of `width`:
  // chunk and row of fetch j
  auto mn_row = [&](auto w, auto ni, int j) {
    constexpr int LPR = decltype(w)::value / 8;  // lanes per row
    return (wv * decltype(ni)::value + j) * (kWave / LPR) + lane / LPR;
  };
  auto mn_col = [&](auto w, int row) {
    constexpr int LPR = decltype(w)::value / 8;
    static_assert(LPR >= 16 && LPR <= kWave, "the swizzle moves 8 segments");
    const int c = lane % LPR;
    return ((((c >> 1) ^ mn_swz(row)) << 1) | (c & 1)) * 8;
  };
  using WR = std::integral_constant<int, C::RT ? C::BM : 128>;
  using WF = std::integral_constant<int, C::BN>;
  using NR = std::integral_constant<int, C::RI>;
  using NF = std::integral_constant<int, C::FI>;
  if constexpr (C::RT) {
    rs.step = C::SR * g.N * 2;
#pragma unroll
    for (int j = 0; j < C::RI; ++j) {
      const int row = mn_row(WR{}, NR{}, j), col = m0 + mn_col(WR{}, row);
      rs.off[j] = col < g.N ? row : kNever;
      rs.p[j] = g.r + (static_cast<int64_t>(ga + row) * g.N + col) * 2;
    }
  } else {
    rs.step = C::SB;
#pragma unroll
    for (int j = 0; j < C::RI; ++j) {
      const int row = ((wv * C::RI + j) * (kWave / C::CPR) + lane / C::CPR) % C::BM;
      const int chunk = kc_slot<C::SB>(row, lane % C::CPR) << 4;
      int64_t src = -1;
      if (m0 + row < mend) src = C::K == kInput ? m0 + row : source_row(g, m0 + row);
      rs.off[j] = src >= 0 ? chunk : kNever;
      rs.p[j] = g.r + src * red_bytes + chunk;
    }
    if constexpr (C::F8) {
      const int64_t src = t < C::BM && m0 + t < mend ? source_row(g, m0 + t) : -1;
      if (src >= 0) {
        sp = reinterpret_cast<const uint8_t*>(g.r_scale + src * stages);
        sstep = 4;
      }
    }
  }
  // integers: a row's and a column's scale a thread, on their way during the loop
  float row_scale = 0.0f, col_scale = 0.0f;
  if constexpr (C::I8) {
    static_assert(C::BM <= C::Threads && C::BN <= C::Threads, "a thread per row and column");
    const int64_t src = t < C::BM && m0 + t < mend ? source_row(g, m0 + t) : -1;
    if (src >= 0) row_scale = g.r_scale[src];
    if (t < C::BN && n0 + t < g.N)
      col_scale = g.f_scale[static_cast<int64_t>(e) * g.N + n0 + t];
  }
  // gathered F: the next stage's entries of rows, this wavefront's consecutive
  // ones
  constexpr int kWaveRows = C::K == kWeightsBy ? C::FBytes / (C::BN * 2) / C::Waves : 1;
  uint32_t next_row[kWaveRows];
  auto load_rows = [&](int stage) {
#pragma unroll
    for (int j = 0; j < kWaveRows; ++j) {
      const int k = stage * C::SR + wv * kWaveRows + j;
      next_row[j] = k < red ? static_cast<uint32_t>(((const_i32*)g.rows)[ga + k]) : ~0u;
    }
  };
  if constexpr (C::FT) {
    fs.step = C::SR * g.K * 2;
#pragma unroll
    for (int j = 0; j < C::FI; ++j) {
      const int row = mn_row(WF{}, NF{}, j), col = n0 + mn_col(WF{}, row);
      fs.off[j] = col < g.K ? row : kNever;
      if (C::K == kWeightsBy)
        fs.p[j] = g.f + static_cast<int64_t>(col) * 2;
      else
        fs.p[j] = g.f + (C::K == kInput ? e * wsz : 0) +
                  (static_cast<int64_t>(C::K == kInput ? row : ga + row) * g.K + col) * 2;
    }
  } else {
    fs.step = C::SB;
#pragma unroll
    for (int j = 0; j < C::FI; ++j) {
      const int row = (wv * C::FI + j) * (kWave / C::CPR) + lane / C::CPR;
      const int chunk = kc_slot<C::SB>(row, lane % C::CPR) << 4;
      fs.off[j] = n0 + row < g.N ? chunk : kNever;
      fs.p[j] = g.f + e * wsz + static_cast<int64_t>(n0 + row) * red_bytes + chunk;
    }
  }
  // a stage as it lies in its buffer: R, row scales, F
  auto issue_r = [&](int stage, uint32_t lds) {
    if constexpr (C::RT)
      fetch<C::RI, kUnitMN>(rs, stage, red, lds, wv * C::RI, C::RBytes / 1024);
    else
      fetch<C::RI, kUnitK>(rs, stage, red_bytes, lds, wv * C::RI, C::RBytes / 1024);
    if constexpr (C::F8)
      dma4(stage < stages ? sp + stage * sstep : zero_block(),
           lds + C::RBytes + wv * 256);
  };
  auto issue_f = [&](int stage, uint32_t lds) {
    if constexpr (!C::FT) {
      fetch<C::FI, kUnitK>(fs, stage, red_bytes, lds, wv * C::FI, C::FBytes / 1024);
    } else if constexpr (C::K != kWeightsBy) {
      fetch<C::FI, kUnitMN>(fs, stage, red, lds, wv * C::FI, C::FBytes / 1024);
    } else {
#pragma unroll
      for (int j = 0; j < C::FI; ++j) {  // kPer rows per fetch, as many parts of a wavefront
        constexpr int kPer = kWaveRows / C::FI;
        int64_t src = -1;
#pragma unroll
        for (int r = 0; r < kPer; ++r) {
          const uint32_t s = next_row[kPer * j + r];
          const int64_t b = s < g.row_limit ? static_cast<int64_t>(row_div(s, g.div_magic)) : -1;
          if (lane / (kWave / kPer) == r) src = b;
        }
        dma16(fs.off[j] != kNever && src >= 0 ? fs.p[j] + src * g.K * 2 : zero_block(),
              lds + (wv * C::FI + j) * 1024);
      }
      load_rows(stage + 1);
    }
  };
  auto issue = [&](int stage, int buf) {
    issue_r(stage, lds0 + buf * C::Stage);
    issue_f(stage, lds0 + buf * C::Stage + C::RBytes + C::SBytes);
  };
  if constexpr (C::K == kWeightsBy) load_rows(0);

  typename C::Acc acc[C::RF][C::FF];
#pragma unroll
  for (int i = 0; i < C::RF; ++i)
#pragma unroll
    for (int j = 0; j < C::FF; ++j) acc[i][j] = typename C::Acc{0, 0, 0, 0};
  const int mw = wm * C::RF * 16, nw = wn * C::FF * 16;
  const_f32* fsc = nullptr;  // this wavefront's row of weight scales
  float ws_next = 0.0f;      // ... of the next stage
  if constexpr (C::F8) {
    fsc = (const_f32*)(g.f_scale + (static_cast<int64_t>(e) * ((g.N + kBlock - 1) / kBlock) +
                                    min(n0 + nw, g.N - 1) / kBlock) * stages);
    ws_next = fsc[0];
  }

  auto math = [&](int stage, const uint8_t* sr, const uint8_t* sf) {
    if constexpr (C::F8) {
      // a block's product p = sum of 128 codes' products, scaled into acc.  One
      // row of fragments behind the matrix instructions, so that none of them
      // is waited for: row i's instructions, each followed by the scaling of row
      // i - 1, with row i + 1 on its way from LDS.
      const float ws = ws_next;
      ws_next = fsc[min(stage + 1, stages - 1)];
      const float* rsc = reinterpret_cast<const float*>(sr + C::RBytes) + mw + (lane & 15);
      u32x4_t fa[C::FF][2], rb[2][2];
#pragma unroll
      for (int j = 0; j < C::FF; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) fa[j][h] = frag_k<C::SB>(sf, nw + j * 16, h, lane);
#pragma unroll
      for (int h = 0; h < 2; ++h) rb[0][h] = frag_k<C::SB>(sr, mw, h, lane);
      float sc[C::RF];
#pragma unroll
      for (int i = 0; i < C::RF; ++i) sc[i] = rsc[i * 16] * ws;
      f32x4_t p[2][C::FF];
#pragma unroll
      for (int i = 0; i <= C::RF; ++i) {
        const int cur = i & 1, old = cur ^ 1;
        if (i + 1 < C::RF) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            rb[old][h] = frag_k<C::SB>(sr, mw + (i + 1) * 16, h, lane);
        }
#pragma unroll
        for (int j = 0; j < C::FF; ++j) {
          if (i < C::RF) p[cur][j] = codes_product(fa[j], rb[cur]);
          if (i > 0) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              acc[i - 1][j][q] = fmaf(sc[i - 1], p[old][j][q], acc[i - 1][j][q]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
#pragma unroll
      for (int kk = 0; kk < C::KK; ++kk) {
        u32x4_t fa[C::FF];
#pragma unroll
        for (int j = 0; j < C::FF; ++j) {
          if constexpr (C::FT)
            fa[j] = frag_mn<C::BN>(sf, nw + j * 16, kk, lane);
          else
            fa[j] = frag_k<C::SB>(sf, nw + j * 16, kk, lane);
        }
#pragma unroll
        for (int i = 0; i < C::RF; ++i) {
          u32x4_t rb;
          if constexpr (C::RT)
            rb = frag_mn<C::BM>(sr, mw + i * 16, kk, lane);
          else
            rb = frag_k<C::SB>(sr, mw + i * 16, kk, lane);
#pragma unroll
          for (int j = 0; j < C::FF; ++j) acc[i][j] = mma(fa[j], rb, acc[i][j]);
        }
      }
    }
  };

  if constexpr (C::PP) {
    // ---- the loop of the two halves in turn: wavefronts 0..3 and 4..7 (one of
    // each on every SIMD) run half a stage apart, so that while one half's
    // matrix instructions run, the other reads its operands from LDS.  Three
    // stages are in flight; a stage's buffer is fetched into after its last
    // reader has its data.  (64-deep stages with one meeting each, both halves
    // at once: 1.7 us a stage where two of these take 1.5.)
    static_assert(C::KK == 1 && !C::F8, "one matrix instruction a stage");
#pragma unroll
    for (int s = 0; s < C::NST - 1; ++s) issue(s, s);
    wait_and_meet<(C::NST - 2) * C::Fetches>();  // stage 0 is here
    if (wv >= C::Waves / 2) asm volatile("s_barrier" ::: "memory");
    int buf = 0;
    for (int s = 0; s < stages; ++s) {
      const uint8_t* st = smem + buf * C::Stage;
      u32x4_t fa[C::FF], rb[C::RF];
#pragma unroll
      for (int j = 0; j < C::FF; ++j)
        fa[j] = C::FT ? frag_mn<C::BN>(st + C::RBytes + C::SBytes, nw + j * 16, 0, lane)
                      : frag_k<C::SB>(st + C::RBytes + C::SBytes, nw + j * 16, 0, lane);
#pragma unroll
      for (int i = 0; i < C::RF; ++i)
        rb[i] = C::RT ? frag_mn<C::BM>(st, mw + i * 16, 0, lane)
                      : frag_k<C::SB>(st, mw + i * 16, 0, lane);
      issue(s + C::NST - 1, buf == 0 ? C::NST - 1 : buf - 1);
      wait_fetches<(C::NST - 2) * C::Fetches>();  // this wavefront's part of stage s + 1
      reads_and_meet();
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int i = 0; i < C::RF; ++i)
#pragma unroll
        for (int j = 0; j < C::FF; ++j) acc[i][j] = mma(fa[j], rb[i], acc[i][j]);
      __builtin_amdgcn_s_setprio(0);
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("s_barrier" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      buf = buf == C::NST - 1 ? 0 : buf + 1;
    }
    if (wv < C::Waves / 2) asm volatile("s_barrier" ::: "memory");
    wait_and_meet<0>();  // no fetch into LDS outlives the tile
  } else {
    // ---- the loop: NST - 1 stages in flight; one meeting per stage, after
    // which the buffer of the stage before is free
#pragma unroll
    for (int s = 0; s < C::NST - 1; ++s) issue(s, s);
    int buf = 0;
    for (int s = 0; s < stages; ++s) {
      wait_and_meet<(C::NST - 2) * C::Fetches>();
      issue(s + C::NST - 1, buf == 0 ? C::NST - 1 : buf - 1);
      const uint8_t* st = smem + buf * C::Stage;
      math(s, st, st + C::RBytes + C::SBytes);
      buf = buf == C::NST - 1 ? 0 : buf + 1;
    }
    wait_and_meet<0>();  // no fetch into LDS outlives the tile
  }

  // ---- store: a lane holds columns 4 q .. 4 q + 3 of row m of each fragment
  // (q = lane / 16).  float32: 16 bytes each, 64 in a row of the store.  bf16:
  // the odd 16-lane rows of one fragment trade places with the even ones of
  // the next, after which a lane has 8 columns of one of them: 64 bytes in a
  // row again (stores of 8 bytes per lane, 32 in a row, took twice the time).
  const int cols = C::FT ? g.K : g.N;
  const int q = lane >> 4;
  f32x4_t wsc[C::FF];
  float* scales = reinterpret_cast<float*>(smem);  // the rows', the columns'
  if constexpr (C::I8) {
    if (t < C::BM) scales[t] = row_scale;
    if (t < C::BN) scales[C::BM + t] = col_scale;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < C::FF; ++j)
      wsc[j] = *reinterpret_cast<const f32x4_t*>(scales + C::BM + nw + j * 16 + q * 4);
  }
#pragma unroll
  for (int i = 0; i < C::RF; ++i) {
    const int m = m0 + mw + i * 16 + (lane & 15);
    const float xsc = C::I8 ? scales[mw + i * 16 + (lane & 15)] : 1.0f;
    auto value = [&](int j) -> f32x4_t {
      if constexpr (C::I8)
        return __builtin_convertvector(acc[i][j], f32x4_t) * xsc * wsc[j];
      else
        return acc[i][j];
    };
    const int64_t row = (C::DW ? static_cast<int64_t>(e) * g.N + m : m) * cols;
    if (out_f32) {
#pragma unroll
      for (int j = 0; j < C::FF; ++j) {
        const int n = n0 + nw + j * 16 + q * 4;
        if (m < mend && n < cols)
          *reinterpret_cast<f32x4_t*>(static_cast<float*>(out) + row + n) = value(j);
      }
    } else {
#pragma unroll
      for (int j = 0; j < C::FF; j += 2) {
        const f32x4_t u = value(j), v = value(j + 1);
        const auto x = __builtin_amdgcn_permlane16_swap(pack_bf16(u[0], u[1]),
                                                        pack_bf16(v[0], v[1]), false, false);
        const auto y = __builtin_amdgcn_permlane16_swap(pack_bf16(u[2], u[3]),
                                                        pack_bf16(v[2], v[3]), false, false);
        const int n = n0 + nw + (j + (q & 1)) * 16 + (q >> 1) * 8;
        if (m < mend && n < cols)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + row + n) =
              make_uint4(x[0], y[0], x[1], y[1]);
      }
    }
  }
}

// Workgroup -> tile: runs of `run` consecutive tiles go to one XCD (workgroups
// are dealt to the 8 XCDs in turn), so that tiles which share a group's rows
// or weights share an L2.  Long runs share more, short ones balance groups of
// unequal size: 16 where the products bound the call (64 groups of 512 rows,
// 2048 x 2048: 322 us against 336 with 4), 4 elsewhere (the skewed prompt of
// 256 groups over 4096 x 6144: 2437 us against 2529; weight gradients, whose
// groups are seldom even, with runs of 4 / 16: 64 skewed groups of 2048 x 1024
// 268 / 286, gathered 378 / 427, of 2048 x 2048 494 / 510, gathered 677 / 745; 64
// even ones of 2048 x 1024 235 / 223).
constexpr int kXcds = 8, kLongRun = 16, kShortRun = 4;
__device__ __forceinline__ int64_t my_tile(int run) {
  const int xcd = blockIdx.x % kXcds, i = blockIdx.x / kXcds;
  return (static_cast<int64_t>(i / run) * kXcds + xcd) * run + i % run;
}
uint32_t tile_grid(int64_t tiles) {
  constexpr int64_t step = kXcds * kLongRun;  // whole runs of either length
  return static_cast<uint32_t>((tiles + step - 1) / step * step);
}

// Tile r of a group's mt x nt: four row tiles at a time, column by column, so
// that a run of tiles shares both its rows and its weights.
struct Place {
  int m, n;
};
__device__ __forceinline__ Place place(int r, int mt, int nt) {
  constexpr int kHigh = 4;
  const int band = r / (kHigh * nt), h = min(kHigh, mt - band * kHigh), i = r - band * kHigh * nt;
  return {band * kHigh + i % h, i / h};
}
// ... of the tile that find_group found (n = 0: one on its own, at row tile t).
__device__ __forceinline__ Place place(const Group& gr, int col, int nt) {
  return gr.n ? place(gr.t * nt + col, gr.n, nt) : Place{gr.t, col};
}

// Row tiles are 256 high (codes: 128, as both the codes and their bf16 values
// sit in registers; 256 x 128 tiles, two after the other, took 1671 us for the
// skewed prompt and 364 for 64 skewed groups over 2048 x 2048, where these take
// 1612 and 331); a group's last one takes the smallest height that holds its
// rows.  Where bf16 rows left over are at most 64 for each full tile, as many of
// those as it takes are 320 high instead (160 accumulators a lane, 247
// registers): a tile of few rows would read all of the weights once more (64
// groups of about 512 rows over 2048 x 2048 341 us without, 318 with; one of 4200
// rows over 4096 x 4096 161 and 121; the skewed prompt 2440 and 2410).  Codes
// have no registers left for it.  The short ones are bound by their fetches and
// keep three or four stages in LDS.
constexpr int kBN = 256, kThreads = 512, kCus = 256;
template <int KIND>
using T128 = Cfg<KIND, 2, 4, 4, 4, 3>;
template <int KIND>
using Tall = std::conditional_t<KIND == kCodes, T128<KIND>, Cfg<KIND, 2, 4, 8, 4, 4, 64, true>>;
template <int KIND>
using High = Cfg<KIND, 2, 4, 10, 4, 4, 64, true>;
template <int KIND>
using T64 = Cfg<KIND, 1, 8, 4, 2, 3>;
template <int KIND>
using T32 = Cfg<KIND, 1, 8, 2, 2, 4>;

// From this many rows a group on (on average) the products bound the call, and
// the tallest tiles go first, so that the last ones to run are short; below,
// the weights' bytes do, and tiles in the groups' order mix both kinds of work.
constexpr int kTallFirstRows = 192;

constexpr int cmax(int a, int b) { return a > b ? a : b; }
template <class... C>
constexpr int lds_of() {
  int m = 0;
  ((m = cmax(m, C::Lds)), ...);
  return m;
}

template <int KIND>
__global__ __launch_bounds__(kThreads) void grouped_tiles(GroupedMm g) {
  constexpr int kBM = Tall<KIND>::BM;
  constexpr int kExtra = KIND <= kInput || KIND == kInts ? High<KIND>::BM - kBM : 0;
  __shared__ __align__(1024)
      uint8_t smem[lds_of<std::conditional_t<(kExtra > 0), High<KIND>, Tall<KIND>>, T128<KIND>,
                          T64<KIND>, T32<KIND>>()];
  const bool tall_first = g.P >= kTallFirstRows * g.E;
  const int64_t id = my_tile(tall_first ? kLongRun : kShortRun);
  const int nt = ((KIND == kInput ? g.K : g.N) + kBN - 1) / kBN;
  const Group gr =
      find_group<kBM, kThreads, kExtra>(g, id / nt, tall_first, reinterpret_cast<int*>(smem));
  if (gr.e < 0) return;
  const Place at = place(gr, static_cast<int>(id % nt), nt);
  const int m0 = gr.a + at.m * kBM + min(at.m, gr.high) * kExtra, n0 = at.n * kBN;
  const int mend = min(gr.b, m0 + kBM + (at.m < gr.high ? kExtra : 0));
  auto run = [&](auto cfg) {
    tile<decltype(cfg)>(g, smem, gr.e, m0, mend, n0, gr.a, gr.b, g.out, g.out_f32);
  };
  if constexpr (kExtra > 0) {
    if (mend - m0 > kBM) {
      run(High<KIND>{});
      return;
    }
  }
  if (mend - m0 > 128)
    run(Tall<KIND>{});
  else if (mend - m0 > 64)
    run(T128<KIND>{});
  else if (mend - m0 > 32)
    run(T64<KIND>{});
  else
    run(T32<KIND>{});
}

// The gradient's tile of a group without rows: zeros, a row of the tile per
// wavefront (bf16: two).  Through the fragments' stores, of 64 bytes in each of
// 16 rows, 2.2 GB of them took 456 us, so 405.
template <class C>
__device__ void zero_tile(const GroupedMm& g, int e, int m0, int mend, int n0, void* out,
                          bool out_f32) {
  const int size = out_f32 ? 4 : 2, per = 16 / size, lanes = C::BN / per;
  const int c = n0 + static_cast<int>(threadIdx.x) % lanes * per;
  if (c >= g.K) return;
  uint8_t* p = static_cast<uint8_t*>(out) + (static_cast<int64_t>(e) * g.N * g.K + c) * size;
  for (int m = m0 + static_cast<int>(threadIdx.x) / lanes; m < mend; m += C::Threads / lanes)
    *reinterpret_cast<uint4*>(p + static_cast<int64_t>(m) * g.K * size) = make_uint4(0, 0, 0, 0);
}

// Weights' gradients: every group's [N][K], its rows in g.split parts.  One
// part: to dw.  More: float32 sums to workspace[part][E][N][K], joined by
// join_parts.
template <class T, class U>
__device__ __forceinline__ void weight_tile(const GroupedMm& g, uint8_t* smem) {
  const int nt = (g.K + T::BN - 1) / T::BN, mt = (g.N + T::BM - 1) / T::BM;
  const int64_t id = my_tile(kShortRun);
  const int r = static_cast<int>(id % (mt * nt));
  const int e = static_cast<int>(id / (mt * nt) % g.E), z = static_cast<int>(id / (mt * nt) / g.E);
  if (z >= g.split) return;
  int a, b;
  group_bounds(g, e, a, b);
  void* out = g.out;
  bool out_f32 = g.out_f32;
  if (g.split > 1) {
    const int part = ((b - a) / g.split + 64) / 64 * 64;  // whole stages, split parts hold all
    a = min(b, a + z * part);
    b = min(b, a + part);
    out = static_cast<float*>(g.workspace) + static_cast<int64_t>(z) * g.E * g.N * g.K;
    out_f32 = true;
  }
  const Place at = place(r, mt, nt);
  const int m0 = at.m * T::BM, n0 = at.n * T::BN;
  if (a >= b)
    zero_tile<T>(g, e, m0, min(g.N, m0 + T::BM), n0, out, out_f32);
  else if (g.N - m0 > U::BM)
    tile<T>(g, smem, e, m0, g.N, n0, a, b, out, out_f32);
  else
    tile<U>(g, smem, e, m0, g.N, n0, a, b, out, out_f32);
}
template <int KIND>
__global__ __launch_bounds__(kThreads) void grouped_weight_tiles(GroupedMm g) {
  __shared__ __align__(1024) uint8_t smem[lds_of<Tall<KIND>, T128<KIND>>()];
  weight_tile<Tall<KIND>, T128<KIND>>(g, smem);
}

// Few weights (SmallDw): 128 x 128 tiles of four wavefronts, so that fewer
// parts of the rows fill the chip.
template <int KIND>
using SmallDw = Cfg<KIND, 2, 2, 4, 4, 3>;
template <int KIND>
__global__ __launch_bounds__(256) void grouped_weight_small(GroupedMm g) {
  __shared__ __align__(1024) uint8_t smem[SmallDw<KIND>::Lds];
  weight_tile<SmallDw<KIND>, SmallDw<KIND>>(g, smem);
}

// dw = the parts' sum, in their order; four elements per thread.
__global__ __launch_bounds__(256) void join_parts(GroupedMm g) {
  const int64_t n = static_cast<int64_t>(g.E) * g.N * g.K;
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  const float* p = static_cast<const float*>(g.workspace) + i;
  f32x4_t v = *reinterpret_cast<const f32x4_t*>(p);
  for (int z = 1; z < g.split; ++z) v += *reinterpret_cast<const f32x4_t*>(p + z * n);
  if (g.out_f32) {
    *reinterpret_cast<f32x4_t*>(static_cast<float*>(g.out) + i) = v;
  } else {
    const uint2 w = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.out) + i) = w;
  }
}

// How a weight gradient is laid out: 256 x 256 or 128 x 128 tiles, and where
// those are too few for the CUs, each group's rows in as many parts as fill
// them, of 256 rows on average at least.
struct WeightPlan {
  bool small;
  int64_t tiles;  // of one part
  int parts;
  int64_t ns;  // expected
};
// Time of a plan: its rounds of tiles (a row of a tile's contraction takes 30 or
// 11 ns, its ends 5 us), whole ones for one group; with several, which are
// seldom even, their mean and the rest of a group of two and a half times
// that; the parts' sums written and read.  us, 128 x 128 against 256 x 256 tiles: 4096
// rows, 1024 x 1024 27 / 38, 2048 x 2048 54 / 62; 16384 rows, 2560 x 2560 327 /
// 242, 4096 x 3840 653 / 456; 8 groups of 1024 rows, 1024 x 1280 51 / 43, skewed
// 55 / 79; 32 of 512, 512 x 768 35 / 27, skewed 47 / 84; 16 of 2048, skewed,
// 2048 x 1024 231 / 181.  The terms are for ranking the two: what they leave out
// (operands read several times, stores) is alike in both, and adds up to half as
// much again (64 skewed groups of 2048 x 1024: 186 us here, 270 measured).
WeightPlan weight_plan(int E, int P, int N, int K, bool small) {
  using T = Tall<kWeights>;
  using S = SmallDw<kWeights>;
  const int bm = small ? S::BM : T::BM, bn = small ? S::BN : T::BN;
  WeightPlan p{small, static_cast<int64_t>(E) * ((N + bm - 1) / bm) * ((K + bn - 1) / bn), 1, 0};
  const int64_t fill = kCus / p.tiles, mean = P / E;
  const int64_t parts = fill < mean / 256 ? fill : mean / 256;
  if (parts > 1) p.parts = static_cast<int>(parts);
  const int64_t rows_ns = mean / p.parts * (small ? 11 : 30), all = p.tiles * p.parts;
  if (E == 1)
    p.ns = (all + kCus - 1) / kCus * (rows_ns + 5000);
  else
    p.ns = (all > kCus ? all : kCus) * (rows_ns + 5000) / kCus + rows_ns * 3 / 2;
  if (p.parts > 1) p.ns += 3000 + static_cast<int64_t>(E) * N * K * p.parts * 8 / 4500;
  return p;
}
WeightPlan weight_plan(int E, int P, int N, int K) {
  const WeightPlan a = weight_plan(E, P, N, K, false), b = weight_plan(E, P, N, K, true);
  return b.ns < a.ns ? b : a;
}

// Few tiles (narrow outputs, one group of middling size): 64 x 128 tiles of
// four wavefronts, two workgroups per CU.  us, against the large tiles, by
// their number: 36 tiles (1 group of 2048 rows, 1024 x 1024) 13.7 / 33.7, 72
// (8 groups, 512 x 2048) 28.7 / 54.3, 144 (2048 x 2048) 53.0 / 55.6, 272 (one
// group of 4096 rows, 4096 x 2048) 97 / 67.
constexpr int kSmallTiles = 160;
template <int KIND>
using Small = Cfg<KIND, 2, 2, 2, 4, 3>;
template <int KIND>
__global__ __launch_bounds__(256, 2) void grouped_small(GroupedMm g) {
  using T = Small<KIND>;
  __shared__ __align__(1024) uint8_t smem[lds_of<T>()];
  const int nt = ((KIND == kInput ? g.K : g.N) + T::BN - 1) / T::BN;
  const int64_t id = my_tile(kShortRun);
  const Group gr = find_group<T::BM, 256>(g, id / nt, false, reinterpret_cast<int*>(smem));
  if (gr.e < 0) return;
  const Place at = place(gr, static_cast<int>(id % nt), nt);
  const int m0 = gr.a + at.m * T::BM;
  tile<T>(g, smem, gr.e, m0, min(gr.b, m0 + T::BM), at.n * T::BN, gr.a, gr.b, g.out, g.out_f32);
}

// The most row tiles of bm rows that any grouping of P rows can have.
int64_t most_row_tiles(const GroupedMm& g, int bm) {
  return g.P / bm + (g.E < g.P ? g.E : g.P);
}

// ---------------------------------------------------------------------------
// A few rows (few_rows): bound by reading the weights once.  A workgroup takes
// 16 columns of one group (codes: 32); its four wavefronts take turns along K
// (256 bytes of a weight row each), load their weights straight into the matrix
// instruction's A registers -- 16 rows x 64 bytes a load, four loads at once --
// and the group's rows of x into its B registers, 16 at a time, and join their
// sums through LDS in a fixed order.  There is nothing to share through LDS, so
// the loads need no barrier, and bf16's 64 registers let a CU hold 32
// wavefronts (eight loads at once and half as many wavefronts: 82 us against
// 74 for one token; non-temporal loads: 90).  e4m3 codes are widened to bf16
// (exact); two fragments of columns share the widening of
// x (8 tokens over 256 experts of 4096 x 6144: 260-277 us, 5.2-5.5 TB/s; one: 333).
// ---------------------------------------------------------------------------

// Against the tiles, us per call, bf16 and codes.  One expert of N = 4096,
// K = 6144: 1 row 17 / 46 and 18 / 46, 32 rows 28 / 48 and 33 / 46, 64 rows
// 51 / 52 and 58 / 47.  64 of N = K = 2048: 32 rows 45 / 58 and 31 / 28, 240 rows
// 108 / 143 and 58 / 59, skewed 93 / 117 and 54 / 53.  256 of 4096 x 6144: 8 rows
// 77 / 76 and 46 / 50, 512 rows 1909 / 1865 and 1012 / 921, skewed 1400 / 1241 and
// 732 / 628.  Drawn sizes (1 to 250 experts, N and K of 64 to 6144, 90 cases): up
// to three times as fast, 10% slower at worst.  Each 16 rows of a group are a pass
// over its weights: where the experts are large and rows crowd, that costs more
// than the tiles' staging, and past about 3 rows a group (64 in one) everywhere
// (256 of 4096 x 6144, 2048 skewed rows of codes 1525 / 993).
bool few_rows(const GroupedMm& g) { return g.P <= 64 + 3 * g.E; }

// Integers, whose tiles read the weights about as fast wherever there are enough
// of them: few rows in few tiles, and a few rows in groups of their own, but not
// where the weight rows lie 4096 bytes apart (16 of them at once, as here, then
// meet in the same channels) nor where a row is hardly one turn long.  us, this
// kernel / the tiles: one expert of N = 4096, K = 6144 (16 tiles) 16 rows 7.7 / 23.0,
// 48 rows 19.6 / 23.1, 64 rows 25.7 / 23.2; 8 rows over 64 of 1024 x 4096 (32 tiles)
// 7.3 / 16.9, over 256 of 1024 x 2048 (32) 7.0 / 10.5; 64 over 256 of 4096 x 6144 (1024
// tiles) 263 / 267, as a layer routes 8 tokens 225 / 232, skewed 141 / 135, 256 over
// them 1051 / 1032, skewed 396 / 329; 40 over 15 of 1784 x 3568 22.5 / 25.1, 64 over 4 of
// 6144 x 2048 13.8 / 11.2; 8 over 16 of 4096 x 4096 (128 tiles) 29.4 / 22.2; 64 over 256 of
// 1024 x 512 10.9 / 7.0.
bool few_integer_rows(const GroupedMm& g) {
  if ((g.E < g.P ? g.E : g.P) * ((g.N + kBN - 1) / kBN) <= 64) return g.P <= 48;
  return g.P <= 64 && g.P <= 3 * g.E && g.K % 4096 != 0 && g.K >= 1024;
}

constexpr int kSkinnyThreads = 256;
constexpr int kSkinnyWaves = kSkinnyThreads / kWave;

// Expert of the slot-th group that holds rows (each wavefront for itself).
__device__ __forceinline__ int find_slot(const GroupedMm& g, int slot, int lane) {
  for (int e0 = 0; e0 < g.E; e0 += kWave) {
    const int e = e0 + lane;
    int a = 0, b = 0;
    if (e < g.E) group_bounds(g, e, a, b);
    uint64_t m = __ballot(b > a);
    const int n = __popcll(m);
    if (slot < n) {
      for (; slot > 0; --slot) m &= m - 1;
      return e0 + __ffsll(static_cast<unsigned long long>(m)) - 1;
    }
    slot -= n;
  }
  return -1;
}

template <int KIND>
struct Skinny {
  static constexpr bool F8 = KIND == kCodes, I8 = KIND == kInts;
  static constexpr int kFrags = F8 ? 2 : 1;  // fragments of 16 columns per wavefront
  static constexpr int kCols = 16 * kFrags;
  static constexpr int kChunk = F8 || I8 ? 16 : 8;  // contraction elements per lane and load
  static constexpr int kLoads = 4;            // loads per turn and fragment
  static constexpr int kOcc = F8 ? 4 : 8;     // wavefronts per SIMD: 64 registers for bf16
  static constexpr int kSpan = kLoads * kChunk * 4;  // contraction elements of a turn
};

template <int KIND>
__global__ __launch_bounds__(kSkinnyThreads, Skinny<KIND>::kOcc) void grouped_skinny(GroupedMm g,
                                                                                   int nb) {
  using C = Skinny<KIND>;
  constexpr bool F8 = C::F8;
  using Acc = std::conditional_t<C::I8, i32x4_t, f32x4_t>;
  using Sum = std::conditional_t<C::I8, int, float>;
  __shared__ Sum part[kSkinnyWaves][16][C::kCols + 1];
  const int t = threadIdx.x, lane = t & (kWave - 1), wv = t / kWave;
  const int e = __builtin_amdgcn_readfirstlane(find_slot(g, blockIdx.x / nb, lane));
  if (e < 0) return;
  int a, b;
  group_bounds(g, e, a, b);
  const int n0 = (blockIdx.x % nb) * C::kCols, elem = F8 || C::I8 ? 1 : 2;
  const int i16 = lane & 15, q = lane >> 4;
  const int64_t ld = static_cast<int64_t>(g.K) * elem;
  const uint8_t* wp[C::kFrags];
#pragma unroll
  for (int f = 0; f < C::kFrags; ++f)  // columns past N repeat the last
    wp[f] = g.f + (static_cast<int64_t>(e) * g.N + min(n0 + f * 16 + i16, g.N - 1)) * ld + q * 16;
  const int kb = (g.K + kBlock - 1) / kBlock;
  const float* ws = F8 ? g.f_scale + (static_cast<int64_t>(e) * ((g.N + kBlock - 1) / kBlock) +
                                      n0 / kBlock) * kb
                       : nullptr;
  for (int m0 = a; m0 < b; m0 += 16) {
    int64_t src = -1;
    if (m0 + i16 < b) src = source_row(g, m0 + i16);
    const uint8_t* xp = g.r + (src < 0 ? 0 : src) * ld + q * 16;
    Acc acc[C::kFrags];
#pragma unroll
    for (int f = 0; f < C::kFrags; ++f) acc[f] = Acc{0, 0, 0, 0};
    for (int k0 = wv * C::kSpan; k0 < g.K; k0 += kSkinnyWaves * C::kSpan) {
      u32x4_t w[C::kFrags][C::kLoads], x[C::kLoads];
#pragma unroll
      for (int u = 0; u < C::kLoads; ++u) {
        const int k = k0 + u * 4 * C::kChunk;
        const bool in = k + q * C::kChunk < g.K;
        x[u] = u32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int f = 0; f < C::kFrags; ++f) {
          w[f][u] = u32x4_t{0, 0, 0, 0};
          if (in)
            w[f][u] = *reinterpret_cast<const u32x4_t*>(wp[f] + static_cast<int64_t>(k) * elem);
        }
        if (in && src >= 0)
          x[u] = *reinterpret_cast<const u32x4_t*>(xp + static_cast<int64_t>(k) * elem);
      }
      if constexpr (F8) {
#pragma unroll
        for (int h = 0; h < C::kLoads / 2; ++h) {
          const int blk = k0 / kBlock + h;
          if (blk >= kb) break;
          const float s = ws[blk] * (src >= 0 ? g.r_scale[src * kb + blk] : 0.0f);
          f32x4_t p[C::kFrags];
#pragma unroll
          for (int f = 0; f < C::kFrags; ++f) p[f] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int u = 2 * h; u < 2 * h + 2; ++u)
#pragma unroll
            for (int v = 0; v < 4; v += 2) {
              const bf16x8_t xb = codes_to_bf16(x[u][v], x[u][v + 1]);
#pragma unroll
              for (int f = 0; f < C::kFrags; ++f)
                p[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    codes_to_bf16(w[f][u][v], w[f][u][v + 1]), xb, p[f], 0, 0, 0);
            }
#pragma unroll
          for (int f = 0; f < C::kFrags; ++f)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[f][j] = fmaf(s, p[f][j], acc[f][j]);
        }
      } else {
#pragma unroll
        for (int u = 0; u < C::kLoads; ++u)
#pragma unroll
          for (int f = 0; f < C::kFrags; ++f) acc[f] = mma(w[f][u], x[u], acc[f]);
      }
    }
#pragma unroll
    for (int f = 0; f < C::kFrags; ++f)
#pragma unroll
      for (int j = 0; j < 4; ++j) part[wv][i16][f * 16 + q * 4 + j] = acc[f][j];
    __syncthreads();
#pragma unroll
    for (int o = t; o < 16 * C::kCols; o += kSkinnyThreads) {
      const int m = m0 + o / C::kCols, n = n0 + o % C::kCols;
      if (m >= b || n >= g.N) continue;
      Sum sum = 0;
#pragma unroll
      for (int w = 0; w < kSkinnyWaves; ++w) sum += part[w][o / C::kCols][o % C::kCols];
      float v = static_cast<float>(sum);
      if constexpr (C::I8) {
        const int64_t from = source_row(g, m);
        v = v * (from >= 0 ? g.r_scale[from] : 0.0f) *
            g.f_scale[static_cast<int64_t>(e) * g.N + n];
      }
      const int64_t at = static_cast<int64_t>(m) * g.N + n;
      if (g.out_f32)
        static_cast<float*>(g.out)[at] = v;
      else
        static_cast<uint16_t*>(g.out)[at] = f32_to_bf16(v);
    }
    __syncthreads();
  }
}

}  // namespace

size_t grouped_dw_workspace(int E, int P, int N, int K) {
  const int parts = weight_plan(E, P, N, K).parts;
  return parts > 1 ? static_cast<size_t>(parts) * E * N * K * sizeof(float) : 0;
}

hipError_t launch_grouped_mm(const GroupedMm& args, GroupedKind kind, hipStream_t stream) {
  GroupedMm g = args;
  auto go = [&](auto kernel, int64_t tiles, int threads) {
    return launch(kernel, dim3(tile_grid(tiles)), dim3(threads), 0, stream, g);
  };
  if (kind == kGroupedWeights) {
    const WeightPlan p = weight_plan(g.E, g.P, g.N, g.K);
    g.split = p.parts;
    const int64_t tiles = p.tiles * p.parts;
    const hipError_t e =
        p.small ? (g.rows ? go(grouped_weight_small<kWeightsBy>, tiles, 256)
                          : go(grouped_weight_small<kWeights>, tiles, 256))
                : (g.rows ? go(grouped_weight_tiles<kWeightsBy>, tiles, kThreads)
                          : go(grouped_weight_tiles<kWeights>, tiles, kThreads));
    if (e != hipSuccess || g.split == 1) return e;
    const int64_t n = static_cast<int64_t>(g.E) * g.N * g.K;
    return launch(join_parts, dim3(static_cast<uint32_t>((n / 4 + 255) / 256)), dim3(256), 0, stream,
                  g);
  }
  if (kind == kGroupedInts ? few_integer_rows(g) : kind != kGroupedInput && few_rows(g)) {
    auto skinny = [&](auto kernel, int cols) {
      const int nb = (g.N + cols - 1) / cols;
      return launch(kernel, dim3(static_cast<uint32_t>(nb * (g.E < g.P ? g.E : g.P))),
                    dim3(kSkinnyThreads), 0, stream, g, nb);
    };
    switch (kind) {
      case kGroupedRows: return skinny(grouped_skinny<kRows>, Skinny<kRows>::kCols);
      case kGroupedInts: return skinny(grouped_skinny<kInts>, Skinny<kInts>::kCols);
      default: return skinny(grouped_skinny<kCodes>, Skinny<kCodes>::kCols);
    }
  }
  const int cols = kind == kGroupedInput ? g.K : g.N;
  const int bm = kind == kGroupedCodes ? Tall<kCodes>::BM : Tall<kRows>::BM;
  const int64_t tiles = most_row_tiles(g, bm) * ((cols + kBN - 1) / kBN);
  if (tiles < kSmallTiles) {
    using S = Small<kRows>;
    const int64_t small = most_row_tiles(g, S::BM) * ((cols + S::BN - 1) / S::BN);
    switch (kind) {
      case kGroupedRows: return go(grouped_small<kRows>, small, S::Threads);
      case kGroupedInput: return go(grouped_small<kInput>, small, S::Threads);
      case kGroupedInts: return go(grouped_small<kInts>, small, S::Threads);
      default: return go(grouped_small<kCodes>, small, S::Threads);
    }
  }
  switch (kind) {
    case kGroupedRows: return go(grouped_tiles<kRows>, tiles, kThreads);
    case kGroupedInput: return go(grouped_tiles<kInput>, tiles, kThreads);
    case kGroupedInts: return go(grouped_tiles<kInts>, tiles, kThreads);
    default: return go(grouped_tiles<kCodes>, tiles, kThreads);
  }
}

}  // namespace moe
