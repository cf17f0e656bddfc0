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
// M = 128 lanes hold output channels and its N = 16..256 columns hold the
// tokens of one tile, rounded up to 16.  A group's ragged end so costs at most
// 15 columns instead of a 128-row tile, and few tokens cost few columns, which
// leaves short groups bound by reading the weights.
//
// One persistent CTA per SM walks the tiles w = blockIdx.x, + gridDim.x, ...;
// tile w belongs to the group whose cumulative tile count covers it, found in
// shared memory from the device's offsets (the host never waits for them).
// Warp 0 copies (TMA, 128-byte swizzle), warp 1 issues tcgen05.mma kind::i8
// and owns TMEM, warps 2-9 write the results.  Two 256-column accumulators
// let the next tile's products run while the epilogue drains the last one.
// Every mbarrier wait is bounded.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "sm100.cuh"

namespace llmint8 {
namespace product {

constexpr int BM = 128;            // MMA M: channels (TMEM lanes) of a tile
constexpr int BK = 128;            // bytes of K per k-block
constexpr int MAX_BT = 256;        // most tokens of a tile (MMA N)
constexpr int KPB_MAX = 4;         // k-blocks per stage
constexpr int MAX_STAGES = 12;
constexpr int MAX_GROUPS = 1024;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 64 + 32 * EPI_WARPS;
constexpr int TMEM_COLS = 512;     // two accumulators of MAX_BT columns
constexpr int RING_BYTES = 192 * 1024;  // stages, and 16 KiB past the last one (see SLACK)
// A tile of fewer than 128 weight rows is multiplied as 128: the lanes past
// its end read whatever follows in shared memory and are never stored.
constexpr int SLACK_BYTES = BM * BK;
constexpr int SX_BYTES = 2 * MAX_BT * 4;
constexpr int GROUP_BYTES = 2 * (MAX_GROUPS + 1) * 4;
constexpr int BAR_BYTES = 512;
constexpr int SMEM_BYTES = 1024 + RING_BYTES + SLACK_BYTES + SX_BYTES + GROUP_BYTES + BAR_BYTES;
static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");

enum : int { kF16 = 0, kBF16 = 1, kF32 = 2 };

struct Params {
  int S, N, K;         // rows of Xq and Y, weight rows of a group, columns
  int No;              // columns of Y: N, or N / 2 when gated
  int E;               // groups
  const int32_t* offsets;  // [E + 1] on the device, null: one group [0, S)
  int KB, KPB, NU;     // k-blocks, k-blocks per stage, stages per tile
  int ksplit;          // 1: the copies see K as [K / 128][128] (K % 128 == 0); 0: as one row, KPB = 1
  int H;               // weight rows of a tile (a multiple of 8; of 32 when gated)
  int nN;              // tiles along the channels
  int BT;              // most tokens of a tile, a multiple of 16
  int box;             // token rows of one copy; BT is a multiple of it
  int stages;
  const float* sx;
  const float* sw;
  const float* bias;   // null: none
  void* Y;
  uint64_t wait_ns;
};

// A tile: `tok` tokens from row m0 of Xq / Y, weight rows (or gated channel
// pairs) from tile nt of group e.
struct Tile {
  int e, m0, tok, nt;
};

// Tiles of a group of m rows along its tokens, and rows of each (a multiple of
// 16, so that the group's tiles are equal but for the last).
__device__ __forceinline__ int token_tiles(int m, int bt) { return (m + bt - 1) / bt; }

__device__ __forceinline__ Tile find_tile(const Params& p, const int* off, const int* cum, int w) {
  int lo = 0, hi = p.E;  // cum[lo] <= w < cum[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cum[mid] <= w)
      lo = mid;
    else
      hi = mid;
  }
  const int begin = off[lo], m = off[lo + 1] - begin;
  const int mt = token_tiles(m, p.BT);
  const int per = ((m + mt - 1) / mt + 15) / 16 * 16;
  const int r = w - cum[lo];
  Tile t;
  t.e = lo;
  t.nt = r / mt;
  const int i = r - t.nt * mt;
  t.m0 = begin + i * per;
  t.tok = min(per, m - i * per);
  return t;
}

// The groups' bounds and cumulative tile counts, by one warp.  Bounds that
// fall outside [0, S] or run backwards are clamped (no row outside Xq or Y is
// touched) and recorded in the error word.
__device__ __forceinline__ void scan_groups(const Params& p, int* off, int* cum) {
  const int lane = static_cast<int>(lane_id());
  if (!p.offsets) {
    if (lane == 0) {
      off[0] = 0;
      off[1] = p.S;
      cum[0] = 0;
      cum[1] = token_tiles(p.S, p.BT) * p.nN;
    }
    return;
  }
  int base = 0, prev = 0;  // tiles and upper bound of the groups before this chunk
  bool bad = false;
  if (lane == 0) {
    const int o = p.offsets[0];
    prev = min(max(o, 0), p.S);
    bad = prev != o;
    off[0] = prev;
    cum[0] = 0;
  }
  prev = __shfl_sync(0xffffffffu, prev, 0);
  for (int g0 = 0; g0 < p.E; g0 += 32) {
    const int g = g0 + lane;
    const int o = g < p.E ? p.offsets[g + 1] : 0;
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
    int n = g < p.E ? token_tiles(end - begin, p.BT) * p.nN : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, n, d);
      if (lane >= d) n += v;
    }
    if (g < p.E) {
      off[g + 1] = end;
      cum[g + 1] = base + n;
    }
    base += __shfl_sync(0xffffffffu, n, 31);
    prev = __shfl_sync(0xffffffffu, end, 31);
  }
  if (bad && blockIdx.x == 0) atomicOr(&g_error_word, kErrBadIndex);
}

// silu(g) * u in binary32.
__device__ __forceinline__ float gate(float g, float u) { return __fdiv_rn(g, 1.0f + expf(-g)) * u; }

template <int OT>
__device__ __forceinline__ void store_out(void* Y, int64_t i, float v) {
  if constexpr (OT == kF16)
    static_cast<__half*>(Y)[i] = __float2half_rn(v);
  else if constexpr (OT == kBF16)
    static_cast<__nv_bfloat16*>(Y)[i] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(Y)[i] = v;
}

// GATED: the weight copies interleave 16 gate rows with the 16 value rows of
// the same channels, so that lanes l and l + 16 of a warp hold the two halves
// of one output.  OT: output type.
template <bool GATED, int OT>
__global__ void __launch_bounds__(THREADS, 1)
    product_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                   const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* sx_s = reinterpret_cast<float*>(smem + RING_BYTES + SLACK_BYTES);  // [2][MAX_BT]
  int* off = reinterpret_cast<int*>(sx_s + 2 * MAX_BT);                     // [E + 1]
  int* cum = off + MAX_GROUPS + 1;                                          // [E + 1]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SMEM_BYTES - 1024 - BAR_BYTES);
  uint64_t* empty = full + MAX_STAGES;
  uint64_t* tfull = empty + MAX_STAGES;  // [2]
  uint64_t* tempty = tfull + 2;          // [2]
  uint64_t* done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);

  const int warp = static_cast<int>(warp_id());
  const int lane = static_cast<int>(lane_id());

  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tmap_w);
    prefetch_tensormap(&tmap_x);
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], EPI_WARPS);
    }
    mbar_init(done, 1);
    fence_barrier_init();
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  // The codes, scales and offsets may come from the kernel before this one,
  // and so may the weights (a user may have quantised them just now): nothing
  // is read before that kernel is done.  Only then may the next one start, so
  // that a kernel two calls later never runs beside one two calls earlier.
  pdl_wait();
  pdl_launch_dependents();
  if (warp == 2) scan_groups(p, off, cum);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int total = cum[p.E];
  const int a_bytes = p.H * BK, b_bytes = p.BT * BK;  // of one k-block
  const int stage_bytes = (a_bytes + b_bytes) * p.KPB;
  auto stage_b = [&](int s) { return smem + s * stage_bytes; };
  auto stage_a = [&](int s) { return smem + s * stage_bytes + p.KPB * b_bytes; };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int w = blockIdx.x; ok && w < total; w += gridDim.x) {
        const Tile t = find_tile(p, off, cum, w);
        const int boxes = (t.tok + p.box - 1) / p.box;
        const uint32_t tx = static_cast<uint32_t>(p.KPB * (a_bytes + boxes * p.box * BK));
        for (int u = 0; u < p.NU; ++u, ++it) {
          const int s = it % p.stages;
          if (it >= p.stages &&
              !mbar_wait(&empty[s], ((it / p.stages) & 1) ^ 1, p.wait_ns, kErrTimeoutProducer)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[s], tx);
          const int kb = p.ksplit ? u * p.KPB : 0, x = p.ksplit ? 0 : u * BK;
          if constexpr (GATED)
            tma_load_5d(stage_a(s), &tmap_w, &full[s], x, 0, 2 * t.e, t.nt * (p.H / 32), kb);
          else
            tma_load_4d(stage_a(s), &tmap_w, &full[s], x, t.nt * p.H, kb, t.e);
          for (int b = 0; b < boxes; ++b)
            tma_load_3d(stage_b(s) + b * p.box * BK, &tmap_x, &full[s], x, t.m0 + b * p.box, kb);
        }
      }
      // Leave no copy in flight: wait for the last loads of every stage.
      for (int i = it < p.stages ? 0 : it - p.stages; i < it; ++i)
        mbar_wait(&full[i % p.stages], (i / p.stages) & 1, p.wait_ns, kErrTimeoutProducer);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      int it = 0, tc = 0;
      bool ok = true;
      for (int w = blockIdx.x; ok && w < total; w += gridDim.x, ++tc) {
        const Tile t = find_tile(p, off, cum, w);
        const uint32_t idesc = idesc_i8_s32(BM, (t.tok + 15) / 16 * 16);
        const int buf = tc & 1;
        if (tc >= 2) {
          ok = mbar_wait(&tempty[buf], ((tc >> 1) - 1) & 1, p.wait_ns, kErrTimeoutMma);
          if (!ok) break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + static_cast<uint32_t>(buf * MAX_BT);
        for (int u = 0; u < p.NU; ++u, ++it) {
          const int s = it % p.stages;
          ok = mbar_wait(&full[s], (it / p.stages) & 1, p.wait_ns, kErrTimeoutMma);
          if (!ok) break;
          tc_fence_after();
          const int nkb = min(p.KPB, p.KB - u * p.KPB);
          for (int j = 0; j < nkb; ++j) {
            const uint32_t a0 = smem_addr(stage_a(s)) + static_cast<uint32_t>(j * a_bytes);
            const uint32_t b0 = smem_addr(stage_b(s)) + static_cast<uint32_t>(j * b_bytes);
#pragma unroll
            for (int k = 0; k < BK / 32; ++k)
              mma_i8(d, make_sdesc_k_sw128(a0 + k * 32), make_sdesc_k_sw128(b0 + k * 32), idesc,
                     (u > 0 || j > 0 || k > 0) ? 1u : 0u);
          }
          mma_commit(&empty[s]);
        }
        if (ok) mma_commit(&tfull[buf]);
      }
      mma_commit(done);
      mbar_wait(done, 0, p.wait_ns, kErrTimeoutMma);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;                   // TMEM lane quadrant of this warp
    const int set = (warp - 2) >> 2;          // two sets of 4 warps share the columns
    const int etid = static_cast<int>(threadIdx.x) - 64;
    const int row = q * 32 + lane;            // row of the tile = TMEM lane
    int tc = 0;
    for (int w = blockIdx.x; w < total; w += gridDim.x, ++tc) {
      const Tile t = find_tile(p, off, cum, w);
      const int buf = tc & 1;
      float* sxb = sx_s + buf * MAX_BT;
      // The buffer's readers two tiles ago are past the previous tile's barrier.
      for (int j = etid; j < t.tok; j += 32 * EPI_WARPS) sxb[j] = p.sx[t.m0 + j];
      // This lane's weight row n and output column c (past the end: not stored).
      int n, c;
      if constexpr (GATED) {
        c = t.nt * (p.H / 2) + q * 16 + (lane & 15);
        n = c + (lane >> 4) * p.No;
      } else {
        n = c = t.nt * p.H + row;
      }
      const bool mine = row < p.H && c < p.No;
      const int64_t at = static_cast<int64_t>(t.e) * p.N + n;
      const float sw = mine ? p.sw[at] : 0.0f;
      const float b = mine && p.bias ? p.bias[at] : 0.0f;
      const bool ok = mbar_wait(&tfull[buf], (tc >> 1) & 1, p.wait_ns, kErrTimeoutEpilogue);
      if (!named_barrier_and(1, 32 * EPI_WARPS, ok)) break;  // also: sxb is written
      tc_fence_after();
      const uint32_t addr =
          tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(buf * MAX_BT);
      if (q * 32 < p.H) {
        for (int c0 = set * 32; c0 < t.tok; c0 += 64) {
          uint32_t r[32];
          tmem_ld32(addr + c0, r);
          tmem_ld_wait();
          tmem_regs_ready(r);
          const int cnt = min(32, t.tok - c0);
          if constexpr (GATED) {
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const float v0 = static_cast<float>(static_cast<int32_t>(r[j])) * sxb[c0 + j] * sw + b;
              const float v1 = static_cast<float>(static_cast<int32_t>(r[j + 1])) * sxb[c0 + j + 1] * sw + b;
              // Lane l < 16 keeps its gate of column j and takes the value
              // from lane l + 16, which takes the gate of column j + 1.
              const float other = __shfl_xor_sync(0xffffffffu, lane < 16 ? v1 : v0, 16);
              const float y = lane < 16 ? gate(v0, other) : gate(other, v1);
              const int jj = j + (lane >> 4);
              if (mine && jj < cnt) store_out<OT>(p.Y, static_cast<int64_t>(t.m0 + c0 + jj) * p.No + c, y);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float y = static_cast<float>(static_cast<int32_t>(r[j])) * sxb[c0 + j] * sw + b;
              if (mine && j < cnt) store_out<OT>(p.Y, static_cast<int64_t>(t.m0 + c0 + j) * p.No + c, y);
            }
          }
        }
      }
      // This warp has read its columns: the MMAs of the tile after next may
      // write them.
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[buf]);
    }
  }

  // Bring the warps whose lane 0 ran a role back together before the barrier.
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

}  // namespace product
}  // namespace llmint8
