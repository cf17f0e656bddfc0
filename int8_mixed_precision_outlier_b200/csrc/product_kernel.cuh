// product_kernel.cuh -- the product of int8 codes with token and channel
// scales, dense or grouped by expert with ragged sizes:
//
//   z[t, n] = (sum_k Xq[t, k] * Wq[e, n, k]) * sx[t] * sw[e, n] (+ b[e, n])
//   y[t, n] = z[t, n]                                   plain
//   y[t, j] = silu(z[t, j]) * z[t, F + j], N = 2 F      gated
//
// for the rows t of group e: offsets[e] <= t < offsets[e + 1] (dense: one
// group with every row).  '三、模型量化' (lowentro.cn) Q2: r' = s * q on each
// operand; 'LLM quantization, part 2' (hncyxsy.com) §2.1: one scale per
// output channel of W.  The int32 sums are exact; scales, bias and gate are
// applied in binary32 and the result is rounded once to the output type.
//
// The operands are swapped (A = weight rows, B = token codes): the MMA's
// M = 128 lanes hold output channels and its N = 32..256 columns hold the
// tokens of one tile, rounded up to 32 (kind::i8 on a CTA pair takes N in steps
// of 32).  A group's ragged end so costs at most 31 columns instead of a
// 128-row tile, and few tokens cost few columns, which leaves short groups
// bound by reading the weights.
//
// One persistent pair of CTAs per two SMs walks the tiles w = unit, + units,
// ...; tile w belongs to the group whose cumulative tile count covers it, found
// in shared memory from the device's offsets (the host never waits for them).
// Warp 0 copies (TMA, 128-byte swizzle), warp 1 issues tcgen05.mma kind::i8
// and owns TMEM, warps 2-17 write the results, warp 18 plans the tiles.  Two
// 256-column accumulators let the next tile's products run while the epilogue
// drains the last one.  Every mbarrier wait is bounded.
//
// Few tokens are bound by reading the weights (1 x 11008 x 4096: 10.9 us, 45 MB
// at 4.1 TB/s with the launch and the last tiles in it), many by the tensor
// cores (4096 x 28672 x 8192: 583 us, 3.3 POP/s; 654 us sustained, at the card's
// 1000 W).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "sm100.cuh"

namespace llmint8 {
namespace product {

constexpr int BM = 128;            // MMA M: channels (TMEM lanes) of a tile
constexpr int BK = 128;            // bytes of K per k-block
constexpr int MAX_BT = 256;        // most tokens of a tile (MMA N)
constexpr int COL_STEP = 32;       // N of kind::i8 with cta_group::2: 32, 64, ... 256
constexpr int KPB_MAX = 4;         // k-blocks per stage
constexpr int MAX_STAGES = 12;
constexpr int MAX_GROUPS = 1024;   // 32 * 32: see Walk::search
constexpr int EPI_WARPS = 16;
constexpr int PLAN_WARP = 2 + EPI_WARPS;
constexpr int THREADS = 32 * (PLAN_WARP + 1);
constexpr int AHEAD = 8;           // tiles that the planning warp may be ahead of the slowest reader
constexpr int TMEM_COLS = 512;     // two accumulators of MAX_BT columns
constexpr int RING_BYTES = 208 * 1024;
constexpr int SX_BYTES = 2 * MAX_BT * 4;
constexpr int GROUP_BYTES = (2 * (MAX_GROUPS + 1) * 4 + MAX_GROUPS * 4 + MAX_GROUPS * 2 + 15) / 16 * 16;
constexpr int BAR_BYTES = 512;     // barriers, and behind them the tile ring
constexpr int TILES_AT = 384;
static_assert((2 * MAX_STAGES + 5 + 2 * AHEAD) * 8 + 4 <= TILES_AT && TILES_AT + 16 * AHEAD <= BAR_BYTES, "layout");
constexpr int SMEM_BYTES = 1024 + RING_BYTES + SX_BYTES + GROUP_BYTES + BAR_BYTES;
static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
static_assert((RING_BYTES + SX_BYTES + GROUP_BYTES + TILES_AT) % 16 == 0, "the tile ring holds int4");
// A tile of fewer than 128 weight rows is multiplied as 128: the lanes past its
// end, which are never stored, read whatever follows in shared memory, after
// the last stage these tables.
static_assert(SX_BYTES + GROUP_BYTES + BAR_BYTES >= BM * BK, "the last stage's 128 rows end inside shared memory");

enum : int { kF16 = 0, kBF16 = 1, kF32 = 2 };

// A group of m rows is cut into mt = ceil(m / BT) tiles of `per` rows (a
// multiple of COL_STEP, at most BT; the last tile may be shorter).  BT <= 256 is the
// same for all, so the division is a multiplication: with `shift` = 31 +
// ceil(log2 BT) and magic = floor(2^shift / BT) + 1, the product x * magic of
// x = m + BT - 1 < 2^31 exceeds 2^shift x / BT by at most x < 2^shift / BT, so
// the quotient is exact; it stays below 2^64.
struct TileCount {
  uint64_t magic;
  int shift, bt;
};
__host__ inline TileCount tile_count(int bt) {
  int shift = 31;
  while ((1 << (shift - 31)) < bt) ++shift;
  return TileCount{(1ull << shift) / static_cast<uint64_t>(bt) + 1, shift, bt};
}
__host__ __device__ inline int token_tiles(int m, const TileCount& c) {
  return static_cast<int>((static_cast<uint64_t>(m) + static_cast<uint64_t>(c.bt - 1)) * c.magic >> c.shift);
}

struct Params {
  int S, N, K;         // rows of Xq and Y, weight rows of a group, columns
  int No;              // columns of Y: N, or N / 2 when gated
  int E;               // groups
  const int32_t* offsets;  // [E + 1] on the device, null: one group [0, S)
  int KB, KPB, NU;     // k-blocks, k-blocks per stage, stages per tile
  int ksplit;          // 1: the copies see K as [K / 128][128] (K % 128 == 0); 0: as one row, KPB = 1
  int H;               // weight rows of a tile and CTA (a multiple of 8; of 32 when gated)
  int nN;              // tiles along the channels (2 H rows each for CTA pairs)
  int BT;              // most tokens of a tile, a multiple of COL_STEP
  int mt, per;         // without offsets: token tiles, rows of each (of each half, where they have two)
  TileCount count;     // of BT
  int drop;            // 1: weights that one tile alone reads leave L2 first
  int quarter;         // token rows of a copy come in 1..4 quarters (a multiple of 8 rows each)
  int b_rows;          // token rows that a k-block of a stage has room for
  int stages;
  const float* sx;
  const float* sw;
  const float* bias;   // null: none
  void* Y;
  uint64_t wait_ns;
};

// Copies of token rows 1, 2, 3 or 4 quarters high, so that a short tile does
// not fetch a full one's rows and every stage still takes one copy of each
// operand (a second one costs the producer about as much as 16 KiB of data).
struct TokenMaps {
  CUtensorMap m[4];
};

// Columns (the MMA's N) of the products of a tile of `tokens` rows.  Each CTA
// of the pair copies half as many token rows.
__host__ __device__ inline int mma_columns(int tokens) { return (tokens + COL_STEP - 1) / COL_STEP * COL_STEP; }

// Equal shares up to the rounding to COL_STEP; an estimate that falls short of m
// is raised (BT itself never does).
__host__ __device__ inline int tile_rows(int m, int mt, int bt) {
  if (mt <= 1) return mma_columns(m);
  const int share = static_cast<int>(static_cast<float>(m) / static_cast<float>(mt)) + 1;
  int per = mma_columns(share);
  if (per > bt) per = bt;
  if (static_cast<int64_t>(per) * mt < m) per += COL_STEP;
  return per;
}

// Quarters that hold `rows` token rows (1..4).
__host__ __device__ inline int quarters_of(int quarter, int rows) {
  return 1 + (rows > quarter) + (rows > 2 * quarter) + (rows > 3 * quarter);
}

// The groups, in shared memory.
struct Groups {
  int* off;        // [E + 1] rows
  int* cum;        // [E + 1] tiles before the group
  int* mt;         // [E]
  uint16_t* per;   // [E]
};

// a / b for 0 <= a < 2^20, b >= 1: (a + 1/2) / b is at least 1 / (2 b) away
// from every integer, and the two approximate steps are off by less than
// (a + 1) / b * 2^-21.
__device__ __forceinline__ int small_div(int a, int b) {
  return __float2int_rz(__fdividef(static_cast<float>(a) + 0.5f, static_cast<float>(b)));
}

// The tiles w = unit, unit + units, ... of a CTA pair, walked by one warp.  Within a group the
// token tiles of one weight tile come one after the other (the weights are
// then read from L2); moving on needs no division of large numbers: only the
// step `units` and the rest below it are divided.
struct Walk {
  int w, total, units;
  int g, r, mt, nt, i;     // group, tile within it, its token tiles; r = nt * mt + i
  int dq, dr;              // units / mt, units % mt
  int begin, rows, per, tiles;

  __device__ void enter(const Groups& s, int group) {
    g = group;
    begin = s.off[g];
    rows = s.off[g + 1] - begin;
    mt = s.mt[g];
    per = s.per[g];
    tiles = s.cum[g + 1] - s.cum[g];
    r = w - s.cum[g];
    nt = small_div(r, mt);
    i = r - nt * mt;
    dq = small_div(units, mt);
    dr = units - dq * mt;
  }
  // The group whose tiles hold w (cum[g] <= w < cum[g + 1]), by the whole warp:
  // first the 32 groups it is among, then the group, 32 counts at a time.
  __device__ void search(const Params& p, const Groups& s) {
    const int lane = static_cast<int>(lane_id());
    const int block = __popc(__ballot_sync(0xffffffffu, (lane + 1) * 32 < p.E && s.cum[min((lane + 1) * 32, p.E)] <= w));
    const int g0 = block * 32 + lane + 1;
    enter(s, block * 32 + __popc(__ballot_sync(0xffffffffu, g0 < p.E && s.cum[min(g0, p.E)] <= w)));
  }
  __device__ Walk(const Params& p, const Groups& s, int unit, int step) {
    w = unit;
    units = step;
    total = s.cum[p.E];
    if (w < total) search(p, s);
  }
  __device__ bool more() const { return w < total; }
  __device__ void next(const Params& p, const Groups& s) {
    w += units;
    r += units;
    if (r < tiles) {
      nt += dq;
      i += dr;
      if (i >= mt) {
        i -= mt;
        ++nt;
      }
    } else if (w < total) {
      search(p, s);
    }
  }
  // Group, tile along the channels, first row of Xq / Y, rows (negative where the
  // weights leave L2 first); `half` 0 or 1 of a tile of two.
  __device__ int4 tile(const Params& p, bool wide, int half) const {
    const int at = ((i << wide) + half) * per, tokens = min(per, rows - at);
    return make_int4(g, nt, begin + at, p.drop && mt == 1 ? -tokens : tokens);
  }
};

// Fills the groups' tables, by one warp.  Bounds that fall outside [0, S] or
// run backwards are clamped (no row outside Xq or Y is touched) and recorded
// in the error word.
__device__ __forceinline__ void scan_groups(const Params& p, const Groups& s) {
  const int lane = static_cast<int>(lane_id());
  if (!p.offsets) {
    if (lane == 0) {
      s.off[0] = 0;
      s.off[1] = p.S;
      s.cum[0] = 0;
      s.cum[1] = p.mt * p.nN;
      s.mt[0] = p.mt;
      s.per[0] = static_cast<uint16_t>(p.per);
    }
    return;
  }
  // The first chunk's bounds are in flight together with the first bound.
  const int first = p.offsets[0];
  int o = lane < p.E ? p.offsets[lane + 1] : 0;
  int base = 0, prev = min(max(first, 0), p.S);  // tiles and upper bound of the groups before this chunk
  bool bad = prev != first;
  if (lane == 0) {
    s.off[0] = prev;
    s.cum[0] = 0;
  }
  for (int g0 = 0; g0 < p.E; g0 += 32) {
    const int g = g0 + lane;
    const int ahead = g + 32 < p.E ? p.offsets[g + 33] : 0;
    int end = g < p.E ? min(max(o, 0), p.S) : 0;
    // a running maximum: no bound lies before an earlier one
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, end, d);
      if (lane >= d) end = max(end, v);
    }
    end = max(end, prev);
    bad |= g < p.E && end != o;
    int begin = __shfl_up_sync(0xffffffffu, end, 1);
    if (lane == 0) begin = prev;
    const int mt = token_tiles(end - begin, p.count);
    int n = g < p.E ? mt * p.nN : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, n, d);
      if (lane >= d) n += v;
    }
    if (g < p.E) {
      s.off[g + 1] = end;
      s.cum[g + 1] = base + n;
      s.mt[g] = mt;
      s.per[g] = static_cast<uint16_t>(tile_rows(end - begin, mt, p.BT));
    }
    base += __shfl_sync(0xffffffffu, n, 31);
    prev = __shfl_sync(0xffffffffu, end, 31);
    o = ahead;
  }
  if (bad && blockIdx.x == 0) atomicOr(&g_error_word, kErrBadIndex);
}

// silu(g) * u in binary32, by t = e^-|g|, which neither overflows nor leaves a
// flushed reciprocal: g u / (1 + t) for g >= 0, g t u / (1 + t) below.
// t = 2^h (1 + l ln 2) with h + l = -|g| log2 e: h is the rounded product, l its
// error and the part of log2 e that binary32 drops (a constant in two parts, as
// Cody and Waite's), so the error of h does not grow with g.  In units of
// 2^-24: ex2 is within 2 ulp (4) and its correction rounds once, which counts
// r = 1 / (1 + t) times in t r; 1 + t rounds to r, rcp is within 1 ulp (1 / r,
// as 1/2 <= r <= 1) and three products one rounding each: 6 r + 1 / r + 3 <= 10
// units of |silu(g) u|, and half a step of t and of g t where these are
// subnormal (g < -87.3).  At |g| = 106 t is 0.
__device__ __forceinline__ float gate(float g, float u) {
  constexpr double kLog2e64 = 1.4426950408889634, kLn2 = 0.6931471805599453;  // log2 e, ln 2
  constexpr float kLog2e = static_cast<float>(kLog2e64), kLog2eRest = static_cast<float>(kLog2e64 - kLog2e);
  const float c = fminf(fabsf(g), 106.0f);  // a NaN comes back in the last line
  const float h = c * -kLog2e;
  const float l = fmaf(c, -kLog2eRest, fmaf(c, -kLog2e, -h));
  float p, r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(p) : "f"(h));
  const float t = fmaf(p, l * static_cast<float>(kLn2), p);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + t));
  return (g < 0.0f ? g * t : g) * r * u;
}

// The int32 -> binary32 conversion, rounded once, without the conversion unit:
// the upper 20 bits and the lower 12 become floats by their position in a
// mantissa (both exact) and one fused multiply-add joins them.
__device__ __forceinline__ float to_float(int32_t v) {
  const float hi = __int_as_float((v >> 12) + 0x4B400000) - 12582912.0f;          // 1.5 * 2^23
  const float lo = __uint_as_float((static_cast<uint32_t>(v) & 0xFFFu) | 0x4B000000u) - 8388608.0f;
  return fmaf(hi, 4096.0f, lo);
}

template <int OT>
__device__ __forceinline__ void store_out(void* Y, int64_t i, float v) {
  if constexpr (OT == kF16)
    static_cast<__half*>(Y)[i] = __float2half_rn(v);
  else if constexpr (OT == kBF16)
    static_cast<__nv_bfloat16*>(Y)[i] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(Y)[i] = v;
}

// Two values rounded to a 16-bit type, the first in the low half.
template <int OT>
__device__ __forceinline__ uint32_t pack_two(float a, float b) {
  if constexpr (OT == kF16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// ------------------------------------------------------------ epilogue
// The accumulator has channels along the TMEM lanes and tokens along the
// columns: a lane of a warp holds one channel, and a warp writes 32
// consecutive channels of a token (gated: 16 channels of two tokens) straight
// from its registers.  Shared memory stays out of it: the products read and
// the copies write about all that it can move, and turning the tile around in
// it (for 16 bytes a thread) slowed them down by a quarter of a K = 2048 tile.
//
// In a gated tile lanes 0-15 of a quadrant hold the gates and lanes 16-31 the
// values of the same 16 channels.  Of two tokens, lanes 0-15 take the first:
// they give their gate of the second for the value of the first.
template <bool GATED, int OT>
struct Epilogue {
  static constexpr int CH = GATED ? 16 : 32;  // channels of a warp
  static constexpr int CHUNK = 32;            // tokens at a time

  // Tokens 0 .. cnt - 1 of CHUNK columns; `y`: this lane's channel in the first
  // token's row of Y (gated: in the row of the token it takes first).
  template <bool FULL>
  __device__ static void write(const uint32_t (&r)[CHUNK], const float* sx, float sw, float b, bool mine, int cnt,
                               int lane, uint8_t* y, int64_t row_bytes) {
    const bool upper = lane >= 16;
#pragma unroll
    for (int j0 = 0; j0 < CHUNK; j0 += 4) {
      if (!FULL && j0 >= cnt) break;
      const float4 s4 = *reinterpret_cast<const float4*>(sx + j0);
      const float sv[4] = {s4.x, s4.y, s4.z, s4.w};
      float z[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // A gated output takes two conversions, an exponential and a reciprocal
        // of the one unit that does them 16 a clock: half of the conversions go
        // another way.
        const int32_t acc = static_cast<int32_t>(r[j0 + i]);
        z[i] = (GATED && (i & 1) ? to_float(acc) : static_cast<float>(acc)) * sv[i] * sw + b;
      }
      if constexpr (GATED) {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const float other = __shfl_xor_sync(0xffffffffu, upper ? z[i] : z[i + 1], 16);
          const float v = gate(upper ? other : z[i], upper ? z[i + 1] : other);
          if (mine && (FULL || j0 + i + (upper ? 1 : 0) < cnt)) store_out<OT>(y, 0, v);
          y += 2 * row_bytes;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (mine && (FULL || j0 + i < cnt)) store_out<OT>(y, 0, z[i]);
          y += row_bytes;
        }
      }
    }
  }
};

// GATED: the weight copies interleave 16 gate rows with the 16 value rows of
// the same channels, so that lanes l and l + 16 of a warp hold the two halves
// of one output.  OT: output type.
//
// A 2-CTA cluster works on one tile of 2 H weight rows (tcgen05 cta_group::2,
// M = 256): CTA r holds weight rows H r .. of the tile and half of its tokens
// as operands, and after the products H rows by all tokens in its TMEM.  The
// even CTA's elected thread issues the MMAs; both CTAs' copies complete on its
// `full` barriers, and a stage's or a tile's commit arrives at both CTAs.
// (Single CTAs with tiles of 128 rows were within 3 % of pairs on the smallest
// shapes, up to 27 % behind on others.)
//
// WIDE tiles have two halves of up to MAX_BT tokens, one accumulator
// each: a stage brings the weights once and the token rows of both, and the
// products of both follow.  For the planner and the epilogue the halves are
// two tiles, one after the other.
template <bool GATED, int OT, bool WIDE>
__global__ void __launch_bounds__(THREADS, 1)
    product_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ TokenMaps tmaps_x,
                   const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* sx_s = reinterpret_cast<float*>(smem + RING_BYTES);  // [2][MAX_BT]
  Groups groups;
  groups.off = reinterpret_cast<int*>(sx_s + 2 * MAX_BT);
  groups.cum = groups.off + MAX_GROUPS + 1;
  groups.mt = groups.cum + MAX_GROUPS + 1;
  groups.per = reinterpret_cast<uint16_t*>(groups.mt + MAX_GROUPS);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SMEM_BYTES - 1024 - BAR_BYTES);
  uint64_t* empty = full + MAX_STAGES;
  uint64_t* tfull = empty + MAX_STAGES;  // [2]
  uint64_t* tempty = tfull + 2;          // [2]
  uint64_t* done = tempty + 2;
  uint64_t* planned = done + 1;          // [AHEAD]: a tile is in the ring
  uint64_t* taken = planned + AHEAD;     // [AHEAD]: every reader has it
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(taken + AHEAD);
  int4* tiles = reinterpret_cast<int4*>(reinterpret_cast<uint8_t*>(full) + TILES_AT);  // [AHEAD]

  const int warp = static_cast<int>(warp_id());
  const int lane = static_cast<int>(lane_id());
  const int rank = static_cast<int>(cluster_ctarank());
  const int unit = static_cast<int>(blockIdx.x >> 1);
  const int units = static_cast<int>(gridDim.x >> 1);

  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tmap_w);
    for (int i = 0; i < 4; ++i) prefetch_tensormap(&tmaps_x.m[i]);
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * EPI_WARPS);
    }
    mbar_init(done, 1);
    for (int i = 0; i < AHEAD; ++i) {
      mbar_init(&planned[i], 1);
      mbar_init(&taken[i], 1 + (rank == 0 ? 1 : 0) + EPI_WARPS);  // producer, MMA issuer, epilogue warps
    }
    fence_barrier_init();
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();  // both CTAs' barriers are initialised before a copy or commit reaches them
  // The codes, scales and offsets may come from the kernel before this one,
  // and so may the weights (a user may have quantised them just now): nothing
  // is read before that kernel is done.  Only then may the next one start, so
  // that a kernel two calls later never runs beside one two calls earlier.
  auto previous_done = [&]() {
    pdl_wait();
    pdl_launch_dependents();
  };
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int a_bytes = p.H * BK;                     // of one k-block
  const int b_bytes = p.b_rows * BK;
  const int half_bytes = b_bytes * p.KPB;           // the token rows of a stage (of one half)
  const int stage_bytes = a_bytes * p.KPB + (half_bytes << WIDE);
  auto stage_b = [&](int s) { return smem + s * stage_bytes; };
  auto stage_a = [&](int s) { return smem + s * stage_bytes + (half_bytes << WIDE); };

  // A wait of a whole warp with one outcome: lanes that gave up and lanes that
  // did not would part, and never meet again at a warp-wide step.
  auto all_wait = [&](uint64_t* bar, uint32_t parity, uint32_t code) {
    return __all_sync(0xffffffffu, mbar_wait_stage(bar, parity, p.wait_ns, code)) != 0;
  };

  // The next tile of the ring, for a reader that has had `i` of them: false at
  // the end (or when the wait ran out).
  struct Tile {
    int g, nt, row, tokens;  // group, tile along the channels, first row of Xq / Y, rows
    bool drop;               // its weights leave L2 first
  };
  auto take = [&](int& i, Tile& t) {
    const int slot = i % AHEAD;
    const bool ok = all_wait(&planned[slot], (i / AHEAD) & 1, kErrTimeoutProducer);
    const int4 v = tiles[slot];
    t = Tile{v.x, v.y, v.z, abs(v.w), v.w < 0};
    __syncwarp();  // all lanes have read
    if (lane == 0) mbar_arrive(&taken[slot]);
    ++i;
    return ok && t.g >= 0;
  };

  if (warp == PLAN_WARP) {
    // ------------------------------------------------------------ tile plan
    // One warp works the tiles out ahead of the others.  (With a walk in every
    // role the next tile took the MMA issuer about 1000 cycles, beside the
    // epilogue's warps, with two MMAs in flight.)
    const bool ragged = p.offsets != nullptr;
    if (ragged) previous_done();
    scan_groups(p, groups);
    __syncwarp();
    Walk t(p, groups, unit, units);
    bool ok = true;
    for (int i = 0, half = 0; ok; ++i) {
      const int slot = i % AHEAD;
      ok = i < AHEAD || all_wait(&taken[slot], ((i / AHEAD) & 1) ^ 1, kErrTimeoutProducer);
      const bool more = ok && t.more();
      if (lane == 0) {
        tiles[slot] = more ? t.tile(p, WIDE, half) : make_int4(-1, 0, 0, 0);
        mbar_arrive(&planned[slot]);
      }
      __syncwarp();
      if (!more) break;
      if (i == 0 && !ragged) previous_done();  // without offsets nothing here waits for it
      if (half == WIDE) t.next(p, groups);
      half ^= WIDE;
    }
  } else if (warp == 0) {
    // ------------------------------------------------------------ producer
    // All lanes walk the loop, one waits and issues: its addresses and
    // coordinates are then uniform values.  (With the loop inside `if (lane ==
    // 0)` an MMA took 71 cycles to issue and a stage 300 more, whatever its
    // size.)  The others do not ask the stages' barriers: the one that issues
    // moves them on alone, and a lane that it left behind would find its phase
    // gone by and wait for another.
    const bool issuer = elect_one();
    // Weights that no other tile reads, of a call whose weights are more than L2
    // holds (none would be there at the next call), leave L2 first: 256 tokens
    // to 4 of 32 experts of 4096 x 2048 take 45.0 us, 47.0 without; 500 to 2 of 8
    // of 8192 x 4096 51.4 and 53.4; 150 x 27648 x 5120 29.6 and 30.4.  (Smaller
    // weights that would have stayed: 16 x 4096 x 4096 6.35 with it and without,
    // 6.47 and 6.36 sustained, 32 x 8192 x 4096 8.94 and 8.88.)
    const uint64_t first_out = policy_evict_first();
    previous_done();
    int s = 0;              // the stage to fill next
    uint32_t phase = 1;     // parity its `empty` barrier had on the lap before (passes at once on lap 0)
    bool ok = true;
    int i = 0;
    for (Tile t, t2; ok && take(i, t);) {
      if (WIDE && !take(i, t2)) break;
      const int mine = mma_columns(t.tokens) / 2;  // token rows this CTA copies
      const int wt = 2 * t.nt + rank;             // this CTA's weight rows, in units of H
      const int x0 = t.row + rank * mine;
      const int quarters = quarters_of(p.quarter, mine);
      const CUtensorMap* tmap_x = &tmaps_x.m[quarters - 1];
      const int mine2 = WIDE ? mma_columns(t2.tokens) / 2 : 0, x2 = WIDE ? t2.row + rank * mine2 : 0;
      const int quarters2 = WIDE ? quarters_of(p.quarter, mine2) : 0;
      const uint32_t tx = static_cast<uint32_t>(2 * p.KPB * (a_bytes + (quarters + quarters2) * p.quarter * BK));
      for (int u = 0; u < p.NU; ++u) {
        if (issuer && ok) ok = mbar_wait_stage(&empty[s], phase, p.wait_ns, kErrTimeoutProducer);
        if (issuer && ok) {
          const int kb = p.ksplit ? u * p.KPB : 0, x = p.ksplit ? 0 : u * BK;
          const uint32_t bar = map_shared_rank(&full[s], 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[s], tx);
          if constexpr (GATED) {
            if (t.drop)
              tma_load_5d_pair(stage_a(s), &tmap_w, bar, x, 0, 2 * t.g, wt * (p.H / 32), kb, first_out);
            else
              tma_load_5d_pair(stage_a(s), &tmap_w, bar, x, 0, 2 * t.g, wt * (p.H / 32), kb);
          } else {
            if (t.drop)
              tma_load_4d_pair(stage_a(s), &tmap_w, bar, x, wt * p.H, kb, t.g, first_out);
            else
              tma_load_4d_pair(stage_a(s), &tmap_w, bar, x, wt * p.H, kb, t.g);
          }
          tma_load_3d_pair(stage_b(s), tmap_x, bar, x, x0, kb);
          if constexpr (WIDE) tma_load_3d_pair(stage_b(s) + half_bytes, &tmaps_x.m[quarters2 - 1], bar, x, x2, kb);
        }
        if (++s == p.stages) {
          s = 0;
          phase ^= 1;
        }
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    // Every copy of both CTAs has landed once the MMAs that read it are done:
    // the `done` commit covers that.
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const bool issuer = elect_one();
    previous_done();
    if (rank == 0) {
      const uint32_t ring = sdesc_low(smem_addr(smem)), stage_step = static_cast<uint32_t>(stage_bytes) >> 4;
      const uint32_t half_at = static_cast<uint32_t>(half_bytes) >> 4;
      const uint32_t a_at = half_at << WIDE, a_step = static_cast<uint32_t>(a_bytes) >> 4;
      int s = 0, tc = 0;
      uint32_t phase = 0, stage = ring;  // `stage`: descriptor of the stage's token rows
      bool ok = true, ready = false;
      int i = 0;
      for (Tile t, t2; ok && take(i, t); tc += 1 + WIDE) {
        if (WIDE && !take(i, t2)) break;
        const int cols = mma_columns(t.tokens);
        const uint32_t idesc = idesc_i8_s32(2 * BM, cols);
        // k-blocks of a stage lie as the copy put them: its rows apart
        const uint32_t b_step = static_cast<uint32_t>(quarters_of(p.quarter, cols / 2) * p.quarter * BK) >> 4;
        const int cols2 = WIDE ? mma_columns(t2.tokens) : 0;
        const uint32_t idesc2 = idesc_i8_s32(2 * BM, WIDE ? cols2 : COL_STEP);
        const uint32_t b_step2 = static_cast<uint32_t>(quarters_of(p.quarter, cols2 / 2) * p.quarter * BK) >> 4;
        const int buf = tc & 1;
        if (tc >= 2) {
          ok = __all_sync(0xffffffffu,
                          mbar_wait_stage<true>(&tempty[buf], ((tc >> 1) - 1) & 1, p.wait_ns, kErrTimeoutMma));
          if constexpr (WIDE)
            ok = __all_sync(0xffffffffu,
                            ok && mbar_wait_stage<true>(&tempty[1], ((tc >> 1) - 1) & 1, p.wait_ns, kErrTimeoutMma));
          if (!ok) break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + static_cast<uint32_t>(buf * MAX_BT);
        for (int u = 0; u < p.NU; ++u) {
          if (issuer && ok && !ready) ok = mbar_wait_stage(&full[s], phase, p.wait_ns, kErrTimeoutMma);
          uint64_t* const freed = &empty[s];
          const uint32_t here = stage;
          stage += stage_step;
          if (++s == p.stages) {
            s = 0;
            stage = ring;
            phase ^= 1;
          }
          if (issuer && ok) {
            // Asked now, answered while the products are issued.
            ready = mbar_ready(&full[s], phase);
            tc_fence_after();
            const int nkb = u + 1 < p.NU ? p.KPB : p.KB - u * p.KPB;
            auto products = [&](uint32_t acc, uint32_t blow, uint32_t step, uint32_t id) {
              uint32_t alow = here + a_at, add = u > 0;  // the tile's first product overwrites the accumulator
              for (int j = 0; j < nkb; ++j, alow += a_step, blow += step) {
#pragma unroll
                for (int k = 0; k < BK / 32; ++k) {
                  mma_i8_low_pair(acc, alow + 2 * k, blow + 2 * k, id, add);
                  add = 1;
                }
              }
            };
            products(d, here, b_step, idesc);
            if constexpr (WIDE) products(d + MAX_BT, here + half_at, b_step2, idesc2);
            mma_commit_pair(freed, 0x3);
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (ok && issuer) {
          mma_commit_pair(&tfull[buf], 0x3);
          if constexpr (WIDE) mma_commit_pair(&tfull[1], 0x3);
        }
      }
      // The MMAs (of both CTAs) are complete before the pair meets and TMEM is
      // released.  The odd CTA, which would wait here for the whole call, does
      // at that meeting, which has no limit to run out.
      if (issuer) mma_commit_pair(done, 0x1);
      mbar_wait_stage(done, 0, p.wait_ns, kErrTimeoutMma);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    using Epi = Epilogue<GATED, OT>;
    const int q = warp & 3;                   // TMEM lane quadrant of this warp
    const int set = (warp - 2) >> 2;          // sets of 4 warps take turns at the columns
    const int etid = static_cast<int>(threadIdx.x) - 64;
    const int tile_ch = GATED ? p.H / 2 : p.H;  // channels of this CTA's tile
    // What a tile's outputs need from global memory, fetched while the tile
    // before it is written: a token's scale (one thread each) and this lane's
    // channel scales and biases.  (Fetched at its own turn, it made 3400 cycles
    // between two tiles.)
    struct Ahead {
      int m0, tok, c;  // rows of Y; this lane's channel
      bool some, mine;  // the warp has channels inside Y and the tile; this lane's is one
      float sx, sw, b;
    };
    auto fetch = [&](const Tile& t) {
      Ahead a;
      a.m0 = t.row;
      a.tok = t.tokens;
      const int c0 = q * Epi::CH, ch = GATED ? lane & 15 : lane;
      a.c = (2 * t.nt + rank) * tile_ch + c0 + ch;
      a.some = c0 < tile_ch && a.c - ch < p.No;
      a.mine = c0 + ch < tile_ch && a.c < p.No;
      a.sx = etid < a.tok ? p.sx[a.m0 + etid] : 0.0f;
      const int64_t at = static_cast<int64_t>(t.g) * p.N + a.c + (GATED && lane >= 16 ? p.No : 0);
      a.sw = a.mine ? p.sw[at] : 0.0f;
      a.b = a.mine && p.bias ? p.bias[at] : 0.0f;
      return a;
    };
    static_assert(32 * EPI_WARPS >= MAX_BT, "a thread for each token's scale");
    previous_done();
    int tc = 0, i = 0;
    Tile t;
    Ahead next{};
    bool more = take(i, t);
    if (more) next = fetch(t);
    // All epilogue threads leave together, at the barrier: after the last tile,
    // or when a wait of any of them ran out.
    for (;; ++tc) {
      const Ahead a = next;
      const int buf = tc & 1;
      float* sxb = sx_s + buf * MAX_BT;
      // The buffer's readers two tiles ago are past the previous tile's barrier.
      if (more && etid < a.tok) sxb[etid] = a.sx;
      // One thread polls, the others sleep at the barrier.
      const bool ok =
          more && (etid != 0 || mbar_wait_stage(&tfull[buf], (tc >> 1) & 1, p.wait_ns, kErrTimeoutEpilogue));
      if (!named_barrier_and(1, 32 * EPI_WARPS, ok)) break;  // also: sxb is written
      tc_fence_after();
      more = take(i, t);
      if (more) next = fetch(t);
      const uint32_t addr =
          tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(buf * MAX_BT);
      if (a.some) {
        constexpr int SIZE = OT == kF32 ? 4 : 2;
        const int64_t row_bytes = static_cast<int64_t>(p.No) * SIZE;
        for (int c0 = set * Epi::CHUNK; c0 < a.tok; c0 += EPI_WARPS / 4 * Epi::CHUNK) {
          uint32_t r[Epi::CHUNK];
          __syncwarp();  // the lanes' stores may have parted them
          tmem_ld32(addr + c0, r);
          tmem_ld_wait();
          tmem_regs_ready(r);
          uint8_t* y = static_cast<uint8_t*>(p.Y) + (a.m0 + c0 + (GATED && lane >= 16 ? 1 : 0)) * row_bytes +
                       static_cast<int64_t>(a.c) * SIZE;
          const int cnt = a.tok - c0;
          if (cnt >= Epi::CHUNK)
            Epi::template write<true>(r, sxb + c0, a.sw, a.b, a.mine, cnt, lane, y, row_bytes);
          else
            Epi::template write<false>(r, sxb + c0, a.sw, a.b, a.mine, cnt, lane, y, row_bytes);
        }
      }
      // This warp has read its columns: the MMAs of the tile after next may
      // write them.
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(map_shared_rank(&tempty[buf], 0));
    }
  }

  __syncwarp();
  tc_fence_before();
  // Neither CTA leaves while the other may still signal its barriers or, after
  // a timeout, copies of the pair may still be landing.
  if (threadIdx.x == 0 && pipeline_gave_up()) sleep_ns_bounded(20000);
  __syncwarp();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

}  // namespace product
}  // namespace llmint8
