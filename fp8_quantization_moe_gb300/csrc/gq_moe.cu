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
// lanes of one expert find each other, by a match or by a ballot on every bit
// of its number, and rank themselves, so the sort is stable and its result
// unique.
//
// Bound by latency (65,536 slots are half a megabyte): a warp keeps up to
// kSortHold ids per lane in registers, all loaded at once, for both passes;
// longer segments are read twice, in batches of that size.  65,536 slots of
// 64 experts in 16 blocks: 7.9 us, 8 slots 3.1 us (3.8 launched as a cluster
// of one block).  A segment of 256 slots read 32 at a time in both passes took
// 12.6 us for 65,536 slots in 8 blocks.
constexpr int kSortHold = 8;
// The rows' tokens are written in the order of the rows, through shared
// memory, where a block has no more than kSortStage slots: each store written
// where its slot is found touches 32 sectors, and a block's stores alone would
// take a cycle each.
constexpr int kSortStage = 8192;
// A match takes a step per distinct value, a ballot per bit of the expert's
// number a fixed time: matches up to this many live lanes of a warp.  98,286
// slots with three of four dropped: 8.0 us with matches, 9.3 with ballots;
// 65,536 live slots of 64 experts 9.1 and 7.9.
constexpr int kSortMatch = 16;
constexpr int kSortWarpsMax = 32;
constexpr int kSortClusterMax = 16;  // 8 where a device has no room for 16

struct SortParams {
  const void* ids;
  int32_t* offs;
  int32_t* pos;
  int32_t* token;
  int32_t slots;     // below 2^31 - 4096
  int32_t per_warp;  // slots of a warp's segment, a multiple of 32
  int32_t top_k, experts;
  int32_t bits;      // of an expert's number
  uint32_t magic;    // slot / top_k = slot * magic >> shift
  int32_t shift;
  bool stage;        // token rows go through shared memory
};

// The expert of slot p, or -1.
template <bool kI64>
__device__ __forceinline__ int32_t expert_of(const SortParams& p, int32_t slot, int32_t end) {
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
  grid_wait();
  const int E = p.experts;
  const int warps = blockDim.x >> 5;
  uint32_t* total = smem;          // [E] this block's count of each expert
  uint32_t* first = smem + E;      // [E] the first row of each expert for this block
  uint32_t* local = smem + 2 * E;  // [E] the same among the block's own slots
  uint32_t* count = smem + 3 * E;  // [warps][E]
  int2* staged = reinterpret_cast<int2*>(smem + ((3 + warps) * E + 1) / 2 * 2);  // (row, token)
  __shared__ uint32_t wsum[2][kSortWarpsMax];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = cluster_rank(), nblocks = cluster_size();

  for (int i = threadIdx.x; i < warps * E; i += blockDim.x) count[i] = 0u;
  __syncthreads();
  const int32_t lo = static_cast<int32_t>(
      min((static_cast<int64_t>(rank) * warps + warp) * p.per_warp, static_cast<int64_t>(p.slots)));
  const int32_t hi = lo + min(p.per_warp, p.slots - lo);
  uint32_t* mine = count + warp * E;
  int32_t held[kSortHold];  // the segment's first ids
  for (int32_t s0 = lo; s0 < hi; s0 += 32 * kSortHold) {
    int32_t e[kSortHold];
#pragma unroll
    for (int i = 0; i < kSortHold; ++i) e[i] = expert_of<kI64>(p, s0 + 32 * i + lane, hi);
#pragma unroll
    for (int i = 0; i < kSortHold; ++i)
      if (s0 + 32 * i < hi && e[i] >= 0) atomicAdd(mine + e[i], 1u);
    if (s0 == lo) {
#pragma unroll
      for (int i = 0; i < kSortHold; ++i) held[i] = e[i];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    uint32_t sum = 0;
    for (int w = 0; w < warps; w += 4) {  // the warps are a multiple of four
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = count[(w + i) * E + e];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        count[(w + i) * E + e] = sum;
        sum += c[i];
      }
    }
    total[e] = sum;
  }
  cluster_arrive();
  cluster_wait();
  // the experts in chunks of one per thread: counts of the whole cluster and
  // of the blocks before this one, then a scan over the experts
  uint32_t carry = 0, own_carry = 0;
  for (int base = 0; base < E; base += blockDim.x) {
    const int e = base + threadIdx.x;
    uint32_t before = 0, all = 0, own = 0;
    if (e < E) {
      own = total[e];
      uint32_t v[kSortClusterMax];
#pragma unroll
      for (uint32_t c = 0; c < kSortClusterMax; ++c)
        v[c] = c < nblocks ? ld_cluster_u32(map_cluster(smem_addr(total + e), c)) : 0u;
#pragma unroll
      for (uint32_t c = 0; c < kSortClusterMax; ++c) {
        if (c < rank) before += v[c];
        all += v[c];
      }
    }
    uint32_t x = all, z = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, d);
      const uint32_t w = __shfl_up_sync(0xffffffffu, z, d);
      if (lane >= d) {
        x += y;
        z += w;
      }
    }
    if (lane == 31) {
      wsum[0][warp] = x;
      wsum[1][warp] = z;
    }
    __syncthreads();
    uint32_t up = carry, own_up = own_carry;
    const int used = (min(E - base, static_cast<int>(blockDim.x)) + 31) / 32;
    for (int w = 0; w < used; ++w) {
      const uint32_t a = wsum[0][w], b = wsum[1][w];
      if (w < warp) {
        up += a;
        own_up += b;
      }
      carry += a;
      own_carry += b;
    }
    __syncthreads();
    x += up;
    z += own_up;
    if (e < E) {
      if (rank == 0) p.offs[e] = static_cast<int32_t>(x);
      first[e] = x - all + before;
      local[e] = z - own;
    }
  }
  cluster_arrive();  // this block reads no other block's memory any more
  __syncthreads();
  const uint32_t live = carry;
  for (int32_t s0 = lo; s0 < hi; s0 += 32 * kSortHold) {
    int32_t ids[kSortHold];
#pragma unroll
    for (int i = 0; i < kSortHold; ++i)
      ids[i] = s0 == lo ? held[i] : expert_of<kI64>(p, s0 + 32 * i + lane, hi);
#pragma unroll
    for (int i = 0; i < kSortHold; ++i) {
      if (s0 + 32 * i >= hi) break;  // the whole warp
      const int32_t slot = s0 + 32 * i + lane;
      const int32_t e = ids[i];
      // the lanes with the same expert
      uint32_t peers = __ballot_sync(0xffffffffu, e >= 0);
      if (__popc(peers) <= kSortMatch) {
        peers = __match_any_sync(0xffffffffu, e);
      } else {
        for (int k = 0; k < p.bits; ++k) {
          const bool set = (e >> k) & 1;
          const uint32_t with = __ballot_sync(0xffffffffu, set);
          peers &= set ? with : ~with;
        }
      }
      uint32_t place = 0;
      if (e >= 0) place = mine[e] + __popc(peers & ((1u << lane) - 1u));
      __syncwarp();
      if (e >= 0 && lane == 31 - __clz(peers)) mine[e] += __popc(peers);
      __syncwarp();
      if (slot < hi) {
        const int32_t row = e >= 0 ? static_cast<int32_t>(first[e] + place) : -1;
        p.pos[slot] = row;
        if (e >= 0) {
          const int32_t t =
              static_cast<int32_t>(static_cast<uint64_t>(slot) * p.magic >> p.shift);
          if (p.stage)
            staged[local[e] + place] = make_int2(row, t);
          else
            p.token[row] = t;
        }
      }
    }
  }
  if (p.stage) {
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < own_carry; i += blockDim.x) {
      const int2 v = staged[i];
      p.token[v.x] = v.y;
    }
  }
  const int64_t step = static_cast<int64_t>(nblocks) * blockDim.x;
  for (int64_t r = live + static_cast<int64_t>(rank) * blockDim.x + threadIdx.x; r < p.slots; r += step)
    p.token[r] = -1;
  cluster_wait();
}

// --------------------------------------------------------------- dispatch --
// Rows are handled in 16-byte chunks, one per thread: a row is split into
// equal spans of at most kThreads chunks, so that an odd width leaves no block
// of a few threads.  (Whole rows per block, several chunks per thread, took
// 116 us instead of 92 for the sum below: too few loads in flight.)
constexpr int kThreads = 256;
constexpr int kBatch = 8;  // slots whose loads are in flight together (4 where a token has no more)

struct Spans {
  int32_t count, chunks, threads;  // spans per row, chunks of each, block size
};

Spans spans_of(int32_t chunks) {
  Spans s;
  s.count = (chunks + kThreads - 1) / kThreads;
  s.chunks = (chunks + s.count - 1) / s.count;
  s.threads = (s.chunks + 31) / 32 * 32;
  return s;
}

struct DispatchParams {
  const uint8_t* x;
  uint8_t* out;
  const int32_t* pos;
  int64_t out_rows, ld_bytes;
  int32_t chunks;  // 16-byte chunks per row
  int32_t span;    // chunks of a block
  int32_t top_k;
};

// The sorted rows of a batch of a token's slots, -1 for the dropped ones.
template <int kB>
__device__ __forceinline__ void load_rows(const int32_t* pos, int32_t j0, int32_t top_k,
                                          int64_t rows, int32_t (&r)[kB]) {
#pragma unroll
  for (int j = 0; j < kB; ++j) {
    r[j] = j0 + j < top_k ? __ldg(pos + j0 + j) : -1;
    if (r[j] >= rows) r[j] = -1;
  }
}

// One block per token and span: a chunk is read once and stored to each of
// the token's rows.  8192 tokens of 8 KB to 8 rows each: 92 us, 6.6 TB/s.
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const DispatchParams p) {
  grid_wait();
  const int64_t t = blockIdx.x;
  const int32_t c = blockIdx.y * p.span + threadIdx.x;
  if (static_cast<int32_t>(threadIdx.x) >= p.span || c >= p.chunks) return;
  const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p.x + t * p.ld_bytes) + c);
  for (int32_t j0 = 0; j0 < p.top_k; j0 += kBatch) {
    int32_t r[kBatch];
    load_rows(p.pos + t * p.top_k, j0, p.top_k, p.out_rows, r);
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (r[j] >= 0)
        reinterpret_cast<uint4*>(p.out)[static_cast<int64_t>(r[j]) * p.chunks + c] = v;
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
  int64_t rows;
  int32_t chunks, span, top_k;
};

// One block per token and span; the loads of kBatch slots are in flight
// together, their sum runs in slot order.
template <bool kF32, int kB>
__global__ void __launch_bounds__(kThreads) combine_kernel(const CombineParams p) {
  grid_wait();
  using C = Chunk<kF32>;
  const int64_t t = blockIdx.x;
  const int32_t c = blockIdx.y * p.span + threadIdx.x;
  if (static_cast<int32_t>(threadIdx.x) >= p.span || c >= p.chunks) return;
  float acc[C::kN];
#pragma unroll
  for (int i = 0; i < C::kN; ++i) acc[i] = 0.0f;
  for (int32_t j0 = 0; j0 < p.top_k; j0 += kB) {
    int32_t r[kB];
    load_rows(p.pos + t * p.top_k, j0, p.top_k, p.rows, r);
    uint4 v[kB];
    float w[kB];
#pragma unroll
    for (int j = 0; j < kB; ++j)
      if (r[j] >= 0) {
        v[j] = __ldcs(p.y + static_cast<int64_t>(r[j]) * p.chunks + c);
        w[j] = p.weights != nullptr ? __ldg(p.weights + t * p.top_k + j0 + j) : 1.0f;
      }
#pragma unroll
    for (int j = 0; j < kB; ++j)
      if (r[j] >= 0) {
        float f[C::kN];
        C::unpack(v[j], f);
#pragma unroll
        for (int i = 0; i < C::kN; ++i) acc[i] = __fmaf_rn(w[j], f[i], acc[i]);
      }
  }
  p.out[t * p.chunks + c] = C::pack(acc);
}

// One block per token: a chunk of g is read once per kB slots, whose dot
// products are summed together: in a thread over its chunks, then over the
// warp by halving (a lane keeps half of its values in each step, so eight
// values take nine exchanges), then over the warps.  8192 tokens of 8 KB, 8
// rows each: 174 us, 6.6 TB/s, with three thread blocks per SM, for which a
// thread spills 28 bytes; 183 with the two that its registers would allow, 189
// with four (128 bytes).
template <bool kF32, int kB>
__global__ void __launch_bounds__(kThreads, kB == kBatch ? 3 : 0) combine_backward_kernel(const CombineParams p) {
  using C = Chunk<kF32>;
  __shared__ float part[kThreads / 32][kB];
  grid_wait();
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int32_t j0 = 0; j0 < p.top_k; j0 += kB) {
    int32_t r[kB];
    load_rows(p.pos + t * p.top_k, j0, p.top_k, p.rows, r);
    float w[kB], dot[kB];
#pragma unroll
    for (int j = 0; j < kB; ++j) {
      w[j] = r[j] >= 0 ? __ldg(p.weights + t * p.top_k + j0 + j) : 0.0f;
      dot[j] = 0.0f;
    }
    for (int32_t c = threadIdx.x; c < p.chunks; c += blockDim.x) {
      float g[C::kN];
      uint4 v[kB];
      const uint4 gv = __ldg(p.g + t * p.chunks + c);
#pragma unroll
      for (int j = 0; j < kB; ++j)
        if (r[j] >= 0) v[j] = __ldcs(p.y + static_cast<int64_t>(r[j]) * p.chunks + c);
      C::unpack(gv, g);
#pragma unroll
      for (int j = 0; j < kB; ++j)
        if (r[j] >= 0) {
          float f[C::kN], d[C::kN];
          C::unpack(v[j], f);
#pragma unroll
          for (int i = 0; i < C::kN; ++i) {
            dot[j] = __fmaf_rn(g[i], f[i], dot[j]);
            d[i] = __fmul_rn(w[j], g[i]);
          }
          __stcs(p.out + static_cast<int64_t>(r[j]) * p.chunks + c, C::pack(d));
        }
    }
#pragma unroll
    for (int n = kB / 2, o = 16; n > 0; n >>= 1, o >>= 1) {
      const bool up = (lane & o) != 0;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float give = up ? dot[i] : dot[i + n];
        const float keep = up ? dot[i + n] : dot[i];
        dot[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
    }
    // lane l holds a partial sum of slot j0 + l / (32 / kB)
#pragma unroll
    for (int o = 16 / kB; o > 0; o >>= 1) dot[0] += __shfl_xor_sync(0xffffffffu, dot[0], o);
    if (lane % (32 / kB) == 0) part[warp][lane / (32 / kB)] = dot[0];
    __syncthreads();
    if (threadIdx.x < kB && j0 + static_cast<int32_t>(threadIdx.x) < p.top_k) {
      float sum = 0.0f;
      for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) sum += part[i][threadIdx.x];
      p.dweights[t * p.top_k + j0 + threadIdx.x] = sum;
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------- host --
gq_status setup(DeviceInfo& info) {
  const int most = (3 + kSortWarpsMax) * kMaxGroups * 4 + kSortStage * 8 + 8;
  for (const void* f : {reinterpret_cast<const void*>(sort_kernel<false>),
                        reinterpret_cast<const void*>(sort_kernel<true>)}) {
    gq_status st = check_cuda(
        cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, most),
        "moe_sort: shared memory size");
    if (st != GQ_OK) return st;
    st = check_cuda(cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1),
                    "moe_sort: cluster size");
    if (st != GQ_OK) return st;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kSortClusterMax);
  cfg.blockDim = dim3(kSortWarpsMax * 32);
  cfg.dynamicSmemBytes = most;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = kSortClusterMax;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  const gq_status st = check_cuda(
      cudaOccupancyMaxActiveClusters(&clusters, sort_kernel<true>, &cfg), "moe_sort: clusters");
  info.sort_cluster = clusters > 0 ? kSortClusterMax : 8;
  return st;
}

gq_status launch_sort(const DeviceInfo& info, const void* ids, bool i64, int64_t tokens, int32_t top_k, int32_t experts,
                      int32_t* offs, int32_t* pos, int32_t* token, cudaStream_t stream) {
  SortParams p;
  p.ids = ids;
  p.offs = offs;
  p.pos = pos;
  p.token = token;
  p.slots = static_cast<int32_t>(tokens * top_k);
  p.top_k = top_k;
  p.experts = experts;
  p.bits = 0;
  while ((1 << p.bits) < experts) ++p.bits;
  // exact for slots below 2^31: with 2^l the power of two at or above top_k,
  // magic = ceil(2^(31 + l) / top_k) <= 2^32 - 1 exceeds the quotient by less
  // than 1, so slot * magic / 2^(31 + l) exceeds slot / top_k by less than
  // 2^-l <= 1 / top_k: the whole part is the same
  int l = 0;
  while ((int64_t(1) << l) < top_k) ++l;
  p.shift = 31 + l;
  p.magic = static_cast<uint32_t>(((uint64_t(1) << p.shift) + top_k - 1) / top_k);
  const int64_t groups32 = (static_cast<int64_t>(p.slots) + 31) / 32;  // warps that a slot group each would fill
  // blocks of up to 32 warps, a cluster of up to 16 of them: a warp's two or
  // more groups of 32 slots are worth another block
  const int warps = static_cast<int>(  // a multiple of four
      groups32 < kSortWarpsMax ? (groups32 + 3 < 4 ? 4 : (groups32 + 3) / 4 * 4) : kSortWarpsMax);
  int blocks = 1;
  while (blocks < info.sort_cluster && static_cast<int64_t>(blocks) * warps * 2 <= groups32) blocks *= 2;
  const int64_t nwarps = static_cast<int64_t>(blocks) * warps;
  p.per_warp = static_cast<int32_t>((groups32 + nwarps - 1) / nwarps * 32);
  p.stage = p.per_warp * warps <= kSortStage;
  const size_t smem = static_cast<size_t>(3 + warps) * experts * 4 +
                      (p.stage ? static_cast<size_t>(p.per_warp) * warps * 8 + 8 : 0);
  return launch_chained("moe_sort: launch", i64 ? sort_kernel<true> : sort_kernel<false>, dim3(blocks),
                        warps * 32, smem, stream, blocks, p);
}

gq_status launch_dispatch(const void* x, int64_t tokens, int64_t row_bytes, int64_t ld_bytes,
                          const int32_t* pos, int32_t top_k, int64_t out_rows, void* out,
                          cudaStream_t stream) {
  DispatchParams p;
  p.x = static_cast<const uint8_t*>(x);
  p.out = static_cast<uint8_t*>(out);
  p.pos = pos;
  p.out_rows = out_rows;
  p.ld_bytes = ld_bytes;
  p.chunks = static_cast<int32_t>(row_bytes / 16);
  p.top_k = top_k;
  const Spans spans = spans_of(p.chunks);
  p.span = spans.chunks;
  const dim3 grid(static_cast<unsigned>(tokens), spans.count);
  return launch_chained("moe_dispatch: launch", dispatch_kernel, grid, spans.threads, 0, stream, 1, p);
}

gq_status launch_combine(const void* y, bool f32, int64_t rows, int64_t H, const int32_t* pos,
                         const float* weights, int64_t tokens, int32_t top_k, void* out,
                         cudaStream_t stream) {
  CombineParams p = {};
  p.y = static_cast<const uint4*>(y);
  p.pos = pos;
  p.weights = weights;
  p.out = static_cast<uint4*>(out);
  p.rows = rows;
  p.chunks = static_cast<int32_t>(H / (f32 ? 4 : 8));
  p.top_k = top_k;
  const Spans spans = spans_of(p.chunks);
  p.span = spans.chunks;
  const dim3 grid(static_cast<unsigned>(tokens), spans.count);
  void (*kernel)(CombineParams) =
      f32 ? (top_k <= 4 ? combine_kernel<true, 4> : combine_kernel<true, kBatch>)
          : (top_k <= 4 ? combine_kernel<false, 4> : combine_kernel<false, kBatch>);
  return launch_chained("moe_combine: launch", kernel, grid, spans.threads, 0, stream, 1, p);
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
  p.rows = rows;
  p.chunks = static_cast<int32_t>(H / (f32 ? 4 : 8));
  p.top_k = top_k;
  const int threads = p.chunks > 0 ? spans_of(p.chunks).threads : 32;
  void (*kernel)(CombineParams) =
      f32 ? (top_k <= 4 ? combine_backward_kernel<true, 4> : combine_backward_kernel<true, kBatch>)
          : (top_k <= 4 ? combine_backward_kernel<false, 4> : combine_backward_kernel<false, kBatch>);
  return launch_chained("moe_combine_backward: launch", kernel, dim3(static_cast<unsigned>(tokens)),
                        threads, 0, stream, 1, p);
}

}  // namespace moe
}  // namespace gq
