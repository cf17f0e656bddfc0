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
constexpr int kRowThreads = 256;

// 16 consecutive elements of a row: 32 bytes of a 16-bit type, 64 of binary32.
template <int IT>
struct Chunk {
  uint4 v[IT == kF32 ? 4 : 2];
};

template <int IT>
__device__ __forceinline__ Chunk<IT> load_chunk(const void* row, int c) {
  constexpr int n = IT == kF32 ? 4 : 2;
  Chunk<IT> k;
  const uint4* p = static_cast<const uint4*>(row) + static_cast<int64_t>(c) * n;
#pragma unroll
  for (int i = 0; i < n; ++i) k.v[i] = p[i];
  return k;
}

template <int IT>
__device__ __forceinline__ void widen_chunk(const Chunk<IT>& k, float (&x)[16]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&k);
  if constexpr (IT == kF32) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float2 f;
      if constexpr (IT == kF16)
        f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      else
        f = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

// Magnitudes order like the bits below the sign, NaN above infinity above
// every finite value, so the row maximum is an integer maximum and also tells
// whether the row holds a value that is not finite.
template <int IT>
__device__ __forceinline__ uint32_t chunk_max(const Chunk<IT>& k, uint32_t m) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&k);
  if constexpr (IT == kF32) {
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
  } else {  // two 16-bit maxima side by side
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
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

// Codes of 16 values (quant8's argument in quant.cuh holds for every binary32
// x with |x / s| <= 127 (1 + 2^-22), which a subnormal s still satisfies as
// long as inv is finite; an infinite inv makes d a NaN and takes the division).
__device__ __forceinline__ uint4 quant16(const float (&x)[16], float s, float inv) {
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
  uint32_t tb[16];
  bool near = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float t = __fmaf_rn(x[i], inv, kMagic);
    const float d = __fmaf_rn(x[i], inv, -__fsub_rn(t, kMagic));
    near |= !(fabsf(d) < 0.5f - 0x1p-12f);
    tb[i] = __float_as_uint(t);
  }
  if (near) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float t = __uint_as_float(tb[i]);
      const float d = __fmaf_rn(x[i], inv, -__fsub_rn(t, kMagic));
      if (!(fabsf(d) < 0.5f - 0x1p-12f)) tb[i] = static_cast<uint32_t>(quant_code(x[i], s)) & 0xFFu;
    }
  }
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = __byte_perm(__byte_perm(tb[4 * i], tb[4 * i + 1], 0x0040),
                       __byte_perm(tb[4 * i + 2], tb[4 * i + 3], 0x0040), 0x5410);
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// One CTA per row; thread i takes chunks i, i + blockDim.x, ...  VPT > 0: at
// most VPT chunks a thread, kept in registers between the maximum and the
// codes; VPT = 0: read again (from L1 or L2).  Without positions row t goes to
// row t; with them, to every row positions[t * copies + j] >= 0.
template <int IT, int VPT>
__global__ void __launch_bounds__(kRowThreads) quantize_rows_kernel(const void* X, int K,
                                                                    const int32_t* positions, int copies,
                                                                    int S, int8_t* Xq,
                                                                    float* xscale) {
  __shared__ uint32_t red[kRowThreads / 32];
  // No early trigger: a kernel started early may read these codes as weights.
  pdl_wait();
  const int64_t t = blockIdx.x;
  const int nchunk = K >> 4;
  const uint8_t* row = static_cast<const uint8_t*>(X) + t * K * (IT == kF32 ? 4 : 2);
  Chunk<IT> keep[VPT > 0 ? VPT : 1];
  uint32_t m = 0;
  if constexpr (VPT > 0) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < nchunk) keep[i] = load_chunk<IT>(row, c);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (static_cast<int>(threadIdx.x + i * blockDim.x) < nchunk) m = chunk_max<IT>(keep[i], m);
  } else {
    for (int c = threadIdx.x; c < nchunk; c += blockDim.x) m = chunk_max<IT>(load_chunk<IT>(row, c), m);
  }
  m = __reduce_max_sync(0xffffffffu, widen_max<IT>(m));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) m = max(m, red[i]);
  const bool finite = m < 0x7F800000u;
  const float s = finite ? __fdiv_rn(__uint_as_float(m), 127.0f) : __uint_as_float(0x7FFFFFFFu);
  const float inv = finite ? scale_reciprocal(s) : 0.0f;

  auto put = [&](int c, const uint4& q) {
    if (!positions) {
      reinterpret_cast<uint4*>(Xq + t * K)[c] = q;
      return;
    }
    for (int j = 0; j < copies; ++j) {
      const int r = positions[t * copies + j];
      if (r >= 0 && r < S) reinterpret_cast<uint4*>(Xq + static_cast<int64_t>(r) * K)[c] = q;
    }
  };
  auto code = [&](const Chunk<IT>& k) {
    if (!finite) return make_uint4(0u, 0u, 0u, 0u);
    float x[16];
    widen_chunk<IT>(k, x);
    return quant16(x, s, inv);
  };
  if constexpr (VPT > 0) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < nchunk) put(c, code(keep[i]));
    }
  } else {
    for (int c = threadIdx.x; c < nchunk; c += blockDim.x) put(c, code(load_chunk<IT>(row, c)));
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
// One cluster of 1..8 CTAs: CTA r takes the r-th part of the choices, each of
// its warps a run of consecutive ones.  Pass 1 counts per warp and expert in
// shared memory (one lane per distinct id adds the lanes that match it, so no
// two lanes meet in a counter); the prefix over warps, CTAs (distributed
// shared memory) and experts gives each warp its first position per expert;
// pass 2 hands them out in order.  No atomics: the result does not depend on
// timing.
constexpr int kPosThreads = 1024;
constexpr int kPosWarps = kPosThreads / 32;
constexpr int kPosMaxCtas = 8;

__host__ __device__ constexpr int pos_smem_bytes(int E) { return (kPosWarps + 2) * E * 4; }

template <typename ID>
__global__ void __launch_bounds__(kPosThreads, 1)
    expert_positions_kernel(const ID* ids, int64_t S, int E, int64_t per_warp,
                            int32_t* positions, int32_t* offsets) {
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
  __syncthreads();
  const int64_t begin = (static_cast<int64_t>(rank) * kPosWarps + warp) * per_warp;
  const int64_t end = min(S, begin + per_warp);
  auto key_at = [&](int64_t i) {
    if (i >= end) return -1;
    const ID v = ids[i];
    return v >= 0 && v < static_cast<ID>(E) ? static_cast<int>(v) : -1;
  };
  int* mine = cnt + warp * E;
  for (int64_t i = begin; i < end; i += 32) {
    const int key = key_at(i + lane);
    const uint32_t same = __match_any_sync(0xffffffffu, key);
    if (key >= 0 && lane == __ffs(same) - 1) mine[key] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kPosThreads) {
    int run = 0;
    for (int w = 0; w < kPosWarps; ++w) {
      const int c = cnt[w * E + e];
      cnt[w * E + e] = run;
      run += c;
    }
    tot[e] = run;
  }
  cluster_sync();
  // E <= kPosThreads: one expert per thread.
  int before = 0, all = 0;
  if (static_cast<int>(threadIdx.x) < E) {
    for (int r = 0; r < ctas; ++r) {
      const int c = static_cast<int>(ld_cluster_u32(map_shared_rank(tot + threadIdx.x, static_cast<uint32_t>(r))));
      before += r < rank ? c : 0;
      all += c;
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
  for (int64_t i = begin; i < end; i += 32) {
    const int key = key_at(i + lane);
    const uint32_t same = __match_any_sync(0xffffffffu, key);
    int p = -1;
    if (key >= 0) p = base[key] + mine[key] + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (key >= 0 && lane == __ffs(same) - 1) mine[key] += __popc(same);
    __syncwarp();
    if (i + lane < end) positions[i + lane] = p;
  }
}

// ------------------------------------------------------------ combine
//   out[t, n] = sum_j weights[t, j] * Y[positions[t, j], n]
// over the j with a position, in binary32 and ascending j (one order, so the
// result does not depend on timing), rounded once.  Y's rows are read once
// and 16 bytes at a time where N and the types allow.
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

// VEC: N % 8 == 0, a thread takes 8 consecutive columns.
template <int IT, int OT, bool VEC>
__global__ void __launch_bounds__(kCombineThreads)
    expert_combine_kernel(const void* Y, int S, int N, const int32_t* positions,
                          const float* weights, int k, void* out) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t = blockIdx.x;
  constexpr int W = VEC ? 8 : 1;
  const int n = (blockIdx.y * kCombineThreads + threadIdx.x) * W;
  if (n >= N) return;
  float acc[W];
#pragma unroll
  for (int i = 0; i < W; ++i) acc[i] = 0.0f;
#pragma unroll 4
  for (int j = 0; j < k; ++j) {
    const int r = positions[t * k + j];
    if (r < 0 || r >= S) {
      if (r != -1 && n == 0) atomicOr(&g_error_word, kErrBadIndex);
      continue;
    }
    const float w = weights[t * k + j];
    const int64_t at = static_cast<int64_t>(r) * N + n;
    if constexpr (VEC) {
      if constexpr (IT == kF32) {
        const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(Y) + at);
        const float4 b = reinterpret_cast<const float4*>(static_cast<const float*>(Y) + at)[1];
        const float y[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, y[i], acc[i]);
      } else {
        const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(Y) + at);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 f;
          if constexpr (IT == kF16)
            f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
          else
            f = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
          acc[2 * i] = fmaf(w, f.x, acc[2 * i]);
          acc[2 * i + 1] = fmaf(w, f.y, acc[2 * i + 1]);
        }
      }
    } else {
      acc[0] = fmaf(w, load_one<IT>(Y, at), acc[0]);
    }
  }
  const int64_t o = t * N + n;
  if constexpr (!VEC) {
    product::store_out<OT>(out, o, acc[0]);
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
