// gq_moe.cu -- tokens into expert order and back: the stable sort of the
// tokens' expert choices, the copy of token rows into sorted order, the
// weighted sum of a token's expert rows, and that sum's gradients.
//
//   sort      slot p = t * top_k + j chose expert ids[p]; the live slots (id
//             in [0, E)) are numbered by (id, p): pos[p] is a live slot's
//             sorted row, -1 for the others; offs[e] the end of expert e's
//             rows; token[r] the token of row r, -1 behind the last.
//   dispatch  out[pos[t][j]] = x[t]
//   combine   out[t] = sum_j w[t][j] * y[pos[t][j]]       (w = 1 without weights)
//   backward  dy[pos[t][j]] = w[t][j] * g[t],  dw[t][j] = <g[t], y[pos[t][j]]>
//
// Sums run in fp32, j ascending, one rounding at the end; no result depends
// on the order in which threads run (no floating-point atomics).  A position
// outside the row buffer counts as a dropped slot, so no position can
// address memory out of bounds.
#include <cuda_bf16.h>

#include "gq_device.cuh"
#include "gq_internal.h"
#include "gq_tcgen05.cuh"

namespace gq {
namespace moe {

// --------------------------------------------------------------- the sort --
// A counting sort by one cluster of blocks: every warp owns a contiguous
// segment of the slots and counts its experts in shared memory; the counts
// become each warp's first row of each expert (prefix over the block's
// warps, over the cluster's blocks through distributed shared memory, over
// the experts), and a second pass numbers the slots.  Within 32 slots the
// lanes of one expert rank themselves by __match_any_sync, so the sort is
// stable and its result unique.
constexpr int kSortWarpsMax = 32;
constexpr int kSortClusterMax = 8;  // the portable cluster size

struct SortParams {
  const void* ids;
  int32_t* offs;
  int32_t* pos;
  int32_t* token;
  int64_t slots;
  int64_t per_warp;  // slots of a warp's segment, a multiple of 32
  int32_t top_k, experts;
};

// The expert of slot p, or -1.
template <bool kI64>
__device__ __forceinline__ int32_t expert_of(const SortParams& p, int64_t slot, int64_t end) {
  if (slot >= end) return -1;
  if (kI64) {
    const int64_t id = __ldg(static_cast<const long long*>(p.ids) + slot);
    return id >= 0 && id < p.experts ? static_cast<int32_t>(id) : -1;
  }
  const int32_t id = __ldg(static_cast<const int32_t*>(p.ids) + slot);
  return id >= 0 && id < p.experts ? id : -1;
}

template <bool kI64>
__global__ void __launch_bounds__(kSortWarpsMax * 32) sort_kernel(const SortParams p) {
  extern __shared__ uint32_t smem[];
  const int E = p.experts;
  const int warps = blockDim.x >> 5;
  uint32_t* total = smem;          // [E] this block's count of each expert
  uint32_t* first = smem + E;      // [E] the first row of each expert for this block
  uint32_t* count = smem + 2 * E;  // [warps][E]
  __shared__ uint32_t wsum[kSortWarpsMax + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = cluster_rank(), nblocks = cluster_size();

  for (int i = threadIdx.x; i < warps * E; i += blockDim.x) count[i] = 0u;
  __syncthreads();
  const int64_t lo = (static_cast<int64_t>(rank) * warps + warp) * p.per_warp;
  const int64_t hi = min(lo + p.per_warp, p.slots);
  uint32_t* mine = count + warp * E;
  for (int64_t s = lo + lane; s < hi; s += 32) {
    const int32_t e = expert_of<kI64>(p, s, hi);
    if (e >= 0) atomicAdd(mine + e, 1u);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    uint32_t sum = 0;
    for (int w = 0; w < warps; ++w) {
      const uint32_t c = count[w * E + e];
      count[w * E + e] = sum;
      sum += c;
    }
    total[e] = sum;
  }
  cluster_arrive();
  cluster_wait();
  // the experts in chunks of one per thread: counts of the whole cluster and
  // of the blocks before this one, then a scan over the experts
  uint32_t carry = 0;
  for (int base = 0; base < E; base += blockDim.x) {
    const int e = base + threadIdx.x;
    uint32_t before = 0, all = 0;
    if (e < E) {
      for (uint32_t c = 0; c < nblocks; ++c) {
        const uint32_t v = ld_cluster_u32(map_cluster(smem_addr(total + e), c));
        if (c < rank) before += v;
        all += v;
      }
    }
    uint32_t x = all;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    uint32_t up = carry, sum = 0;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) up += wsum[w];
      sum += wsum[w];
    }
    __syncthreads();
    x += up;
    carry += sum;
    if (e < E) {
      if (rank == 0) p.offs[e] = static_cast<int32_t>(x);
      first[e] = x - all + before;
    }
  }
  cluster_arrive();  // this block reads no other block's memory any more
  __syncthreads();
  const uint32_t live = carry;
  for (int64_t s0 = lo; s0 < hi; s0 += 32) {
    const int32_t e = expert_of<kI64>(p, s0 + lane, hi);
    const uint32_t peers = __match_any_sync(0xffffffffu, e);
    uint32_t row = 0;
    if (e >= 0) row = first[e] + mine[e] + __popc(peers & ((1u << lane) - 1u));
    __syncwarp();
    if (e >= 0 && lane == 31 - __clz(peers)) mine[e] += __popc(peers);
    __syncwarp();
    if (s0 + lane < hi) {
      p.pos[s0 + lane] = e >= 0 ? static_cast<int32_t>(row) : -1;
      if (e >= 0) p.token[row] = static_cast<int32_t>((s0 + lane) / p.top_k);
    }
  }
  const int64_t step = static_cast<int64_t>(nblocks) * blockDim.x;
  for (int64_t r = live + static_cast<int64_t>(rank) * blockDim.x + threadIdx.x; r < p.slots; r += step)
    p.token[r] = -1;
  cluster_wait();
}

// --------------------------------------------------------------- dispatch --
constexpr int kThreads = 256;

struct DispatchParams {
  const uint8_t* x;
  uint8_t* out;
  const int32_t* pos;
  int64_t tokens, out_rows, ld_bytes;
  int32_t chunks;  // 16-byte chunks per row
  int32_t top_k;
};

// One block per token and span of kThreads chunks: a chunk is read once and
// stored to each of the token's rows.
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const DispatchParams p) {
  const int64_t t = blockIdx.x;
  const int32_t c = blockIdx.y * kThreads + threadIdx.x;
  if (c >= p.chunks) return;
  const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p.x + t * p.ld_bytes) + c);
  for (int32_t j = 0; j < p.top_k; ++j) {
    const int64_t r = __ldg(p.pos + t * p.top_k + j);
    if (r < 0 || r >= p.out_rows) continue;
    reinterpret_cast<uint4*>(p.out)[r * p.chunks + c] = v;
  }
}

// ---------------------------------------------------------------- combine --
// A 16-byte chunk as fp32 values and back (bf16: 8 values, fp32: 4).
template <bool kF32>
struct Chunk;

template <>
struct Chunk<false> {
  static constexpr int kN = 8;
  __device__ static __forceinline__ void unpack(uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ static __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <>
struct Chunk<true> {
  static constexpr int kN = 4;
  __device__ static __forceinline__ void unpack(uint4 v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  __device__ static __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};

struct CombineParams {
  const uint4* y;
  const uint4* g;        // backward
  const int32_t* pos;
  const float* weights;  // or nullptr: ones (forward)
  uint4* out;            // forward: (tokens, H); backward: dy (rows, H)
  float* dweights;       // backward
  int64_t tokens, rows;
  int32_t chunks, top_k;
};

template <bool kF32>
__global__ void __launch_bounds__(kThreads) combine_kernel(const CombineParams p) {
  using C = Chunk<kF32>;
  const int64_t t = blockIdx.x;
  const int32_t c = blockIdx.y * kThreads + threadIdx.x;
  if (c >= p.chunks) return;
  float acc[C::kN];
#pragma unroll
  for (int i = 0; i < C::kN; ++i) acc[i] = 0.0f;
  for (int32_t j = 0; j < p.top_k; ++j) {
    const int64_t r = __ldg(p.pos + t * p.top_k + j);
    if (r < 0 || r >= p.rows) continue;
    const float w = p.weights != nullptr ? __ldg(p.weights + t * p.top_k + j) : 1.0f;
    float f[C::kN];
    C::unpack(__ldcs(p.y + r * p.chunks + c), f);
#pragma unroll
    for (int i = 0; i < C::kN; ++i) acc[i] = __fmaf_rn(w, f[i], acc[i]);
  }
  p.out[t * p.chunks + c] = C::pack(acc);
}

// One block per token; the block sums each slot's dot product.
template <bool kF32>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(const CombineParams p) {
  using C = Chunk<kF32>;
  __shared__ float part[kThreads / 32];
  const int64_t t = blockIdx.x;
  for (int32_t j = 0; j < p.top_k; ++j) {
    const int64_t r = __ldg(p.pos + t * p.top_k + j);
    const bool live = r >= 0 && r < p.rows;  // the same in the whole block
    float dot = 0.0f;
    if (live) {
      const float w = __ldg(p.weights + t * p.top_k + j);
      for (int32_t c = threadIdx.x; c < p.chunks; c += kThreads) {
        float g[C::kN], f[C::kN], d[C::kN];
        C::unpack(__ldg(p.g + t * p.chunks + c), g);
        C::unpack(__ldcs(p.y + r * p.chunks + c), f);
#pragma unroll
        for (int i = 0; i < C::kN; ++i) {
          dot = __fmaf_rn(g[i], f[i], dot);
          d[i] = __fmul_rn(w, g[i]);
        }
        p.out[r * p.chunks + c] = C::pack(d);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = dot;
    __syncthreads();
    if (threadIdx.x == 0) {
      float sum = 0.0f;
      for (int i = 0; i < kThreads / 32; ++i) sum += part[i];
      p.dweights[t * p.top_k + j] = sum;
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------- host --
gq_status setup(DeviceInfo& info) {
  (void)info;
  const int most = (2 + kSortWarpsMax) * kMaxGroups * 4;
  gq_status st = check_cuda(cudaFuncSetAttribute(sort_kernel<false>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, most),
                            "moe_sort: shared memory size");
  if (st != GQ_OK) return st;
  return check_cuda(cudaFuncSetAttribute(sort_kernel<true>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, most),
                    "moe_sort: shared memory size");
}

gq_status launch_sort(const void* ids, bool i64, int64_t tokens, int32_t top_k, int32_t experts,
                      int32_t* offs, int32_t* pos, int32_t* token, cudaStream_t stream) {
  SortParams p;
  p.ids = ids;
  p.offs = offs;
  p.pos = pos;
  p.token = token;
  p.slots = tokens * top_k;
  p.top_k = top_k;
  p.experts = experts;
  const int64_t groups32 = (p.slots + 31) / 32;  // warps that a slot group each would fill
  const int warps = static_cast<int>(groups32 < 4 ? 4 : groups32 < kSortWarpsMax ? groups32 : kSortWarpsMax);
  int blocks = 1;
  while (blocks < kSortClusterMax && static_cast<int64_t>(blocks) * warps * 2 <= groups32) blocks *= 2;
  const int64_t nwarps = static_cast<int64_t>(blocks) * warps;
  p.per_warp = (groups32 + nwarps - 1) / nwarps * 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(warps * 32);
  cfg.dynamicSmemBytes = static_cast<size_t>(2 + warps) * experts * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = blocks;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return check_cuda(i64 ? cudaLaunchKernelEx(&cfg, sort_kernel<true>, p)
                        : cudaLaunchKernelEx(&cfg, sort_kernel<false>, p),
                    "moe_sort: launch");
}

gq_status launch_dispatch(const void* x, int64_t tokens, int64_t row_bytes, int64_t ld_bytes,
                          const int32_t* pos, int32_t top_k, int64_t out_rows, void* out,
                          cudaStream_t stream) {
  DispatchParams p;
  p.x = static_cast<const uint8_t*>(x);
  p.out = static_cast<uint8_t*>(out);
  p.pos = pos;
  p.tokens = tokens;
  p.out_rows = out_rows;
  p.ld_bytes = ld_bytes;
  p.chunks = static_cast<int32_t>(row_bytes / 16);
  p.top_k = top_k;
  const dim3 grid(static_cast<unsigned>(tokens), (p.chunks + kThreads - 1) / kThreads);
  dispatch_kernel<<<grid, kThreads, 0, stream>>>(p);
  return check_cuda(cudaGetLastError(), "moe_dispatch: launch");
}

gq_status launch_combine(const void* y, bool f32, int64_t rows, int64_t H, const int32_t* pos,
                         const float* weights, int64_t tokens, int32_t top_k, void* out,
                         cudaStream_t stream) {
  CombineParams p = {};
  p.y = static_cast<const uint4*>(y);
  p.pos = pos;
  p.weights = weights;
  p.out = static_cast<uint4*>(out);
  p.tokens = tokens;
  p.rows = rows;
  p.chunks = static_cast<int32_t>(H / (f32 ? 4 : 8));
  p.top_k = top_k;
  const dim3 grid(static_cast<unsigned>(tokens), (p.chunks + kThreads - 1) / kThreads);
  if (f32)
    combine_kernel<true><<<grid, kThreads, 0, stream>>>(p);
  else
    combine_kernel<false><<<grid, kThreads, 0, stream>>>(p);
  return check_cuda(cudaGetLastError(), "moe_combine: launch");
}

gq_status launch_combine_backward(const void* g, const void* y, bool f32, int64_t rows, int64_t H,
                                  const int32_t* pos, const float* weights, int64_t tokens,
                                  int32_t top_k, void* dy, float* dweights, cudaStream_t stream) {
  CombineParams p = {};
  p.y = static_cast<const uint4*>(y);
  p.g = static_cast<const uint4*>(g);
  p.pos = pos;
  p.weights = weights;
  p.out = static_cast<uint4*>(dy);
  p.dweights = dweights;
  p.tokens = tokens;
  p.rows = rows;
  p.chunks = static_cast<int32_t>(H / (f32 ? 4 : 8));
  p.top_k = top_k;
  if (f32)
    combine_backward_kernel<true><<<static_cast<unsigned>(tokens), kThreads, 0, stream>>>(p);
  else
    combine_backward_kernel<false><<<static_cast<unsigned>(tokens), kThreads, 0, stream>>>(p);
  return check_cuda(cudaGetLastError(), "moe_combine_backward: launch");
}

}  // namespace moe
}  // namespace gq
