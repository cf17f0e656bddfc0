// expert_kernels.cuh -- what stands around the int8 products of
// product_kernel.cuh: the row quantisation (directly, or into the rows that a
// grouped product reads), the order of a router's choices by expert, and the
// weighted sum of the experts' outputs.  All are bound by memory or, for few
// tokens, by latency.  Inputs are read with plain loads after griddepcontrol.
// wait: a read-only (non-coherent) load could be moved in front of it.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "prep_kernels.cuh"
#include "product_kernel.cuh"
#include "quant.cuh"
#include "sm100.cuh"

namespace llmint8 {
namespace expert {

using product::kBF16;
using product::kF16;
using product::kF32;
using product::pack_two;

// ------------------------------------------------------------ row quantisation
// '三、模型量化' (lowentro.cn) Q2, as everywhere in this library: s = max|x| /
// 127, code = rint_even(fl(x / s)), 0 when s == 0.  A row with a NaN or an
// infinity gets s = NaN and codes 0, so that every product of that row is NaN
// and no other row is touched.
constexpr int kRowThreads = 1024;  // the most; the host takes as many as the row needs

// 32 bytes of a row: 16 consecutive elements of a 16-bit type, 8 of binary32.
struct Chunk {
  uint4 v[2];
};
template <int IT>
constexpr int kChunk = IT == kF32 ? 8 : 16;

__device__ __forceinline__ Chunk load_chunk(const uint8_t* row, int c) {
  const uint4* p = reinterpret_cast<const uint4*>(row) + 2 * static_cast<int64_t>(c);
  return Chunk{{p[0], p[1]}};
}

// Magnitudes order like the bits below the sign, NaN above infinity above
// every finite value, so the row maximum is an integer maximum and also tells
// whether the row holds a value that is not finite.
template <int IT>
__device__ __forceinline__ uint32_t chunk_max(const Chunk& k, uint32_t m) {
  const uint32_t w[8] = {k.v[0].x, k.v[0].y, k.v[0].z, k.v[0].w, k.v[1].x, k.v[1].y, k.v[1].z, k.v[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (IT == kF32)
      m = max(m, w[i] & 0x7FFFFFFFu);
    else  // two 16-bit maxima side by side
      m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
  }
  return m;
}

// The largest magnitude of the row as binary32 bits, from a thread's chunk_max.
template <int IT>
__device__ __forceinline__ uint32_t widen_max(uint32_t m) {
  if constexpr (IT == kF32) return m;
  const uint32_t h = max(m & 0xFFFFu, m >> 16);
  if constexpr (IT == kBF16) return h << 16;
  return __float_as_uint(half_bits_to_float(h));
}

// Codes of 4 values in a word, as quant8 (quant.cuh) forms them: its argument
// needs a distance of more than 2^-16 + 2^-25 from the half-integers, so 2^-15
// is asked for here and one element in 16384 is divided.  It holds for every
// binary32 x with |x / s| <= 127 (1 + 2^-22), which a subnormal s still
// satisfies as long as inv is finite; an infinite inv makes d a NaN and takes
// the division.
__device__ __forceinline__ uint32_t quant4(const float (&x)[4], float s, float inv) {
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
  uint32_t tb[4];
  bool near = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float t = __fmaf_rn(x[i], inv, kMagic);
    const float d = __fmaf_rn(x[i], inv, -__fsub_rn(t, kMagic));
    near |= !(fabsf(d) < 0.5f - 0x1p-15f);
    tb[i] = __float_as_uint(t);
  }
  if (near) {  // rare: all four by division
#pragma unroll
    for (int i = 0; i < 4; ++i) tb[i] = static_cast<uint32_t>(quant_code(x[i], s)) & 0xFFu;
  }
  return __byte_perm(__byte_perm(tb[0], tb[1], 0x0040), __byte_perm(tb[2], tb[3], 0x0040), 0x5410);
}

// The codes of a chunk, 4 to a word (binary32: two words).
template <int IT>
__device__ __forceinline__ void code_chunk(const Chunk& k, float s, float inv, uint32_t (&o)[kChunk<IT> / 4]) {
  const uint32_t w[8] = {k.v[0].x, k.v[0].y, k.v[0].z, k.v[0].w, k.v[1].x, k.v[1].y, k.v[1].z, k.v[1].w};
#pragma unroll
  for (int g = 0; g < kChunk<IT> / 4; ++g) {
    float x[4];
    if constexpr (IT == kF32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(w[4 * g + i]);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t u = w[2 * g + i];
        const float2 f = IT == kF16 ? __half22float2(*reinterpret_cast<const __half2*>(&u))
                                    : make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
    o[g] = quant4(x, s, inv);
  }
}

// One CTA per row; thread i takes chunks i, i + blockDim.x, ...  VPT > 0: at
// most VPT chunks a thread, kept in registers between the maximum and the
// codes; VPT = 0: read again (from L1 or L2).  Without positions row t goes to
// row t; with them, to every row positions[t * copies + j] >= 0.
//
// Bound by memory where there are many bytes: 8192 x 4096 binary32 takes 25.6 us
// (6.6 TB/s, the copy rate), 4096 x 8192 fp16 18.9 (5.3 TB/s), 2048 x 4096 fp16
// 7.4 (3.4 TB/s; 5.3 us with the rows in L2), where a row's load, maximum and
// stores, one after the other, count.  40 registers let 1536 threads on an SM;
// a limit of 72 measured the same.
template <int IT, int VPT>
__global__ void __maxnreg__(40)
    quantize_rows_kernel(const void* X, int K, const int32_t* positions, int copies, int S, int8_t* Xq,
                         float* xscale) {
  __shared__ uint32_t red[kRowThreads / 32];
  // No early trigger: a kernel started early may read these codes as weights.
  pdl_wait();
  const int64_t t = blockIdx.x;
  const int nchunk = K / kChunk<IT>;
  const uint8_t* row = static_cast<const uint8_t*>(X) + t * K * (IT == kF32 ? 4 : 2);
  Chunk keep[VPT > 0 ? VPT : 1];
  uint32_t m = 0;
  if constexpr (VPT > 0) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      keep[i] = c < nchunk ? load_chunk(row, c) : Chunk{};
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) m = chunk_max<IT>(keep[i], m);
  } else {
    for (int c = threadIdx.x; c < nchunk; c += blockDim.x) m = chunk_max<IT>(load_chunk(row, c), m);
  }
  m = __reduce_max_sync(0xffffffffu, widen_max<IT>(m));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  const int warps = static_cast<int>(blockDim.x >> 5), lane = static_cast<int>(lane_id());
  m = __reduce_max_sync(0xffffffffu, lane < warps ? red[lane] : 0u);
  const bool finite = m < 0x7F800000u;
  const float s = finite ? __fdiv_rn(__uint_as_float(m), 127.0f) : __uint_as_float(0x7FFFFFFFu);
  const float inv = finite ? scale_reciprocal(s) : 0.0f;

  auto put = [&](int c, const uint32_t (&o)[kChunk<IT> / 4]) {
    auto to = [&](int64_t r) {
      if constexpr (IT == kF32)
        reinterpret_cast<uint2*>(Xq + r * K)[c] = make_uint2(o[0], o[1]);
      else
        reinterpret_cast<uint4*>(Xq + r * K)[c] = make_uint4(o[0], o[1], o[2], o[3]);
    };
    if (!positions) {
      to(t);
      return;
    }
    for (int j = 0; j < copies; ++j) {
      const int r = positions[t * copies + j];
      if (r >= 0 && r < S) to(r);
    }
  };
  auto code = [&](int c, const Chunk& k) {
    uint32_t o[kChunk<IT> / 4] = {};
    if (finite) code_chunk<IT>(k, s, inv, o);
    put(c, o);
  };
  if constexpr (VPT > 0) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < nchunk) code(c, keep[i]);
    }
  } else {
    for (int c = threadIdx.x; c < nchunk; c += blockDim.x) code(c, load_chunk(row, c));
  }
  if (!positions) {
    if (threadIdx.x == 0) xscale[t] = s;
  } else {
    for (int j = threadIdx.x; j < copies; j += blockDim.x) {
      const int r = positions[t * copies + j];
      if (r >= 0 && r < S)
        xscale[r] = s;
      else if (r != -1)
        atomicOr(&g_error_word, kErrBadIndex);
    }
  }
}

// ------------------------------------------------------------ expert positions
// A stable counting sort of the S = T k choices by expert:
//   positions[i] = offsets[id_i] + #{ j < i : id_j = id_i },  -1 where id_i is
//   outside [0, E);  offsets = exclusive prefix sums of the experts' counts.
// One cluster of 1..16 CTAs: CTA r takes the r-th part of the choices, each of
// its warps a run of consecutive ones.  A warp counts its choices per expert in
// shared memory (one lane per distinct id adds the lanes that share it, so no
// two lanes meet in a counter), which also gives each choice its rank among
// the warp's choices of that expert; the prefix over warps, CTAs (distributed
// shared memory) and experts gives the warp's first position per expert.  No
// atomics: the result does not depend on timing.
//
// Bound by latency: the ids are loaded once, all in flight, and stay in
// registers with their ranks (65536 choices of 128 experts: 8.45 us, 8.53 with a
// second pass over the ids; 320000 of 256, which takes it, 28.5).  ITEMS > 0: at
// most ITEMS ids a lane.  ITEMS = 0: any number; the ranks wait in `positions`
// and the ids are read again.
constexpr int kPosThreads = 1024;
constexpr int kPosWarps = kPosThreads / 32;
constexpr int kPosMaxCtas = 16;  // a cluster size that a kernel has to opt in to
constexpr int kPosBits = 11;
static_assert(product::MAX_GROUPS < (1 << kPosBits), "an expert and `none` in kPosBits bits");

__host__ __device__ constexpr int pos_smem_bytes(int E) { return (kPosWarps + 2) * E * 4; }

template <typename ID, int ITEMS>
__global__ void __launch_bounds__(kPosThreads, 1)
    expert_positions_kernel(const ID* ids, int64_t S, int E, int64_t per_warp, int32_t* positions,
                            int32_t* offsets) {
  extern __shared__ int pos_smem[];
  int* cnt = pos_smem;               // [kPosWarps][E]
  int* tot = cnt + kPosWarps * E;    // [E]: this CTA's choices of each expert
  int* base = tot + E;               // [E]: this CTA's first position of each
  __shared__ int scratch[33];
  const int warp = static_cast<int>(warp_id());
  const int lane = static_cast<int>(lane_id());
  const int rank = static_cast<int>(cluster_ctarank());
  const int ctas = static_cast<int>(gridDim.x);
  for (int i = threadIdx.x; i < kPosWarps * E; i += kPosThreads) cnt[i] = 0;
  pdl_wait();
  const int64_t begin = (static_cast<int64_t>(rank) * kPosWarps + warp) * per_warp;
  const int64_t end = min(S, begin + per_warp);
  auto key_of = [&](ID v) { return v >= 0 && v < static_cast<ID>(E) ? static_cast<int>(v) : -1; };
  int* mine = cnt + warp * E;
  // The lanes with this lane's key, by one ballot per bit (match.any compares
  // lane by lane: with it 65536 choices of 128 experts take 10.2 us).
  const int bits = 32 - __clz(E);  // of keys in [0, E), and E for none
  auto alike = [&](int key) {
    const uint32_t k = static_cast<uint32_t>(key >= 0 ? key : E);
    uint32_t same = 0xffffffffu;
#pragma unroll
    for (int b = 0; b < kPosBits; ++b) {
      if (b >= bits) break;
      const uint32_t one = static_cast<uint32_t>(static_cast<int32_t>(k << (31 - b)) >> 31);
      same &= ~(__ballot_sync(0xffffffffu, one != 0u) ^ one);
    }
    return same;
  };
  // The rank of this lane's choice, given the lanes with the same one; counts them.
  auto count = [&](int key, uint32_t same) {
    int r = 0;
    if (key >= 0) r = mine[key];
    __syncwarp();
    if (key >= 0 && lane == __ffs(same) - 1) mine[key] = r + __popc(same);
    __syncwarp();
    return r + __popc(same & ((1u << lane) - 1u));
  };
  int key[ITEMS > 0 ? ITEMS : 1], r[ITEMS > 0 ? ITEMS : 1];
  if constexpr (ITEMS > 0) {
    ID v[ITEMS];  // no branch between the loads: all in flight at once
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) v[i] = begin < end ? ids[min(begin + 32 * i + lane, end - 1)] : static_cast<ID>(-1);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) key[i] = begin + 32 * i + lane < end ? key_of(v[i]) : -1;
    __syncthreads();  // cnt is zero
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) r[i] = count(key[i], alike(key[i]));
  } else {
    __syncthreads();
    for (int64_t i = begin; i < end; i += 32) {
      const int k = i + lane < end ? key_of(ids[i + lane]) : -1;
      const int v = count(k, alike(k));
      if (i + lane < end) positions[i + lane] = v;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kPosThreads) {
    int c[kPosWarps];  // loaded first: a load would wait for the store before it
#pragma unroll
    for (int w = 0; w < kPosWarps; ++w) c[w] = cnt[w * E + e];
    int run = 0;
#pragma unroll
    for (int w = 0; w < kPosWarps; ++w) {
      cnt[w * E + e] = run;
      run += c[w];
    }
    tot[e] = run;
  }
  cluster_sync();
  // E <= kPosThreads: one expert per thread.
  int before = 0, all = 0;
  if (static_cast<int>(threadIdx.x) < E) {
#pragma unroll
    for (int c = 0; c < kPosMaxCtas; ++c) {
      if (c < ctas) {
        const int n = static_cast<int>(ld_cluster_u32(map_shared_rank(tot + threadIdx.x, static_cast<uint32_t>(c))));
        before += c < rank ? n : 0;
        all += n;
      }
    }
  }
  int total;
  const int first = block_exclusive_scan(all, scratch, &total);
  if (static_cast<int>(threadIdx.x) < E) {
    base[threadIdx.x] = first + before;
    if (rank == 0) offsets[threadIdx.x] = first;
  }
  if (rank == 0 && threadIdx.x == 0) offsets[E] = total;
  cluster_sync();  // base is written; no CTA's tot is read any more
  if constexpr (ITEMS > 0) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int64_t at = begin + 32 * i + lane;
      if (at < end) positions[at] = key[i] >= 0 ? base[key[i]] + mine[key[i]] + r[i] : -1;
    }
  } else {
    for (int64_t at = begin + lane; at < end; at += 32) {
      const int k = key_of(ids[at]);
      positions[at] = k >= 0 ? base[k] + mine[k] + positions[at] : -1;
    }
  }
}

// ------------------------------------------------------------ combine
//   out[t, n] = sum_j weights[t, j] * Y[positions[t, j], n]
// over the j with a position, in binary32 and ascending j (one order, so the
// result does not depend on timing), rounded once.  Y's rows are read once
// and 16 bytes at a time where N and the types allow.  Bound by memory: 4096
// tokens of 4 rows of 5120, bf16, take 36.0 us (5.8 TB/s).
constexpr int kCombineThreads = 128;

template <int T>
__device__ __forceinline__ float load_one(const void* p, int64_t i) {
  if constexpr (T == kF16)
    return __half2float(static_cast<const __half*>(p)[i]);
  else if constexpr (T == kBF16)
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  else
    return static_cast<const float*>(p)[i];
}

// VEC: N % 8 == 0, a thread takes 8 consecutive columns; otherwise 8 columns
// kCombineThreads apart, so that as many loads are in flight.
template <int IT, int OT, bool VEC>
__global__ void __launch_bounds__(kCombineThreads)
    expert_combine_kernel(const void* Y, int S, int N, const int32_t* positions, const float* weights, int k,
                          void* out) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t = blockIdx.x;
  const int n = VEC ? (blockIdx.y * kCombineThreads + threadIdx.x) * 8
                    : blockIdx.y * kCombineThreads * 8 + threadIdx.x;
  if (n >= N) return;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
#pragma unroll 4
  for (int j = 0; j < k; ++j) {
    const int r = positions[t * k + j];
    if (r < 0 || r >= S) {
      if (r != -1 && n == 0) atomicOr(&g_error_word, kErrBadIndex);
      continue;
    }
    const float w = weights[t * k + j];
    const int64_t at = static_cast<int64_t>(r) * N + n;
    float y[8];
    if constexpr (!VEC) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        y[i] = n + i * kCombineThreads < N ? load_one<IT>(Y, at + i * kCombineThreads) : 0.0f;
    } else if constexpr (IT == kF32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(Y) + at);
      const float4 a = p[0], b = p[1];
      y[0] = a.x, y[1] = a.y, y[2] = a.z, y[3] = a.w, y[4] = b.x, y[5] = b.y, y[6] = b.z, y[7] = b.w;
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(Y) + at);
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = IT == kF16 ? __half22float2(*reinterpret_cast<const __half2*>(&u[i]))
                                    : make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
        y[2 * i] = f.x;
        y[2 * i + 1] = f.y;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, y[i], acc[i]);
  }
  const int64_t o = t * N + n;
  if constexpr (!VEC) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (n + i * kCombineThreads < N) product::store_out<OT>(out, o + i * kCombineThreads, acc[i]);
  } else if constexpr (OT == kF32) {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(out) + o);
    dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + o) =
        make_uint4(pack_two<OT>(acc[0], acc[1]), pack_two<OT>(acc[2], acc[3]), pack_two<OT>(acc[4], acc[5]),
                   pack_two<OT>(acc[6], acc[7]));
  }
}

}  // namespace expert
}  // namespace llmint8
