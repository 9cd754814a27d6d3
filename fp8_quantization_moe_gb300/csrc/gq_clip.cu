// gq_clip.cu -- the norm over all elements of a list of tensors, and the
// tensors scaled to a largest norm:
//     norm = sqrt(sum of x^2),   y = x * min(1, max_norm / norm)
// Both are streams bound by HBM: the norm reads every element once, the
// scaling reads and writes every element once more.
//
// The tensors are cut into chunks of 16 KB; the blocks of the grid take them in
// turn, each loading its next chunk before it works on the last (without that
// the norm ran at 4.4 TB/s).  The scaling goes through the list backwards: what
// the norm has read last is still in L2.  The table of the tensors comes with the
// launch's parameters: nothing is copied to the device beforehand, so a call
// can be captured.  1.6 GB of bf16: the norm 241 us, 6.7 TB/s; norm and scaling
// to other tensors 742 us.
//
// A thread sums the squares of the 64 bytes that it has of a chunk in fp32, eight
// elements to a partial sum, and everything beyond that in fp64, in an order
// that goes by the sizes and by the addresses within 16 bytes alone: the result
// is the same in every run.  Squares of values past 2^60, or all below 2^-40,
// would leave fp32's range: such a thread squares in fp64.
#include <algorithm>
#include <memory>
#include <new>

#include "gq_tcgen05.cuh"
#include "gq_internal.h"

namespace gq {
namespace clip {

namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;                     // 16-byte vectors per thread and chunk
constexpr int kChunk = kThreads * kVecs * 16;  // bytes
constexpr int kWarps = kThreads / 32;
constexpr int kMostBlocks = 2048;            // partial sums per launch
constexpr int64_t kF32Bit = int64_t(1) << 62;

template <int kCap>
struct Table {
  const uint8_t* in[kCap];
  uint8_t* out[kCap];
  int64_t size[kCap];       // elements, kF32Bit set for fp32
  int32_t first[kCap + 1];  // chunks before each tensor
  int32_t count;
};

// Largest tables; 28 bytes an entry, below the 32 KB of a launch's parameters.
constexpr int kSmall = 16, kLarge = 1024;

// A chunk: `size` bytes per element, `head` single elements up to the first
// 16-byte boundary, `vecs` vectors, `tail` single elements behind them.
struct Chunk {
  const uint8_t* in;
  uint8_t* out;
  int32_t size, head, vecs, tail;
};

template <int kCap>
__device__ __forceinline__ Chunk chunk_of(const Table<kCap>& tab, int32_t c) {
  int32_t lo = 0, hi = tab.count - 1;  // the last tensor whose first chunk is at or before c
  while (lo < hi) {
    const int32_t mid = (lo + hi + 1) >> 1;
    if (tab.first[mid] <= c)
      lo = mid;
    else
      hi = mid - 1;
  }
  Chunk k;
  k.size = (tab.size[lo] & kF32Bit) != 0 ? 4 : 2;
  const int64_t at = static_cast<int64_t>(c - tab.first[lo]) * kChunk;
  const int64_t left = (tab.size[lo] & ~kF32Bit) * k.size - at;
  const int32_t bytes = left < kChunk ? static_cast<int32_t>(left) : kChunk;
  k.in = tab.in[lo] + at;
  k.out = tab.out[lo] + at;
  const int32_t skip =
      min(bytes, static_cast<int32_t>(-static_cast<uint32_t>(reinterpret_cast<uintptr_t>(k.in)) & 15u));
  k.head = skip / k.size;
  k.vecs = (bytes - skip) / 16;
  k.tail = (bytes - skip) % 16 / k.size;
  return k;
}

// This thread's part of a chunk: its vectors, and perhaps a single element.
struct Part {
  uint4 v[kVecs];
  float one;
};

__device__ __forceinline__ float load_one(const uint8_t* p, int32_t size) {
  return size == 4 ? *reinterpret_cast<const float*>(p)
                   : __uint_as_float(uint32_t(*reinterpret_cast<const uint16_t*>(p)) << 16);
}

__device__ __forceinline__ void store_one(uint8_t* p, int32_t size, float v) {
  if (size == 4)
    *reinterpret_cast<float*>(p) = v;
  else
    *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(bf16x2_of(v, 0.0f) & 0xFFFFu);
}

// The place of this thread's single element in bytes, -1 if it has none: at most
// seven at either end, two warps.
__device__ __forceinline__ int32_t single_of(const Chunk& k) {
  const int32_t lane = threadIdx.x & 31;
  if (threadIdx.x < 32) return lane < k.head ? lane * k.size : -1;
  if (threadIdx.x >= 64 || lane >= k.tail) return -1;
  return (k.head + lane) * k.size + k.vecs * 16;
}

__device__ __forceinline__ void load_part(Part& t, const Chunk& k) {
  const uint4* const q = reinterpret_cast<const uint4*>(k.in + k.head * k.size);
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int32_t i = threadIdx.x + j * kThreads;
    t.v[j] = i < k.vecs ? q[i] : make_uint4(0u, 0u, 0u, 0u);
  }
  const int32_t at = single_of(k);
  t.one = at >= 0 ? load_one(k.in + at, k.size) : 0.0f;
}

// The values of a 16-byte vector.
template <int kSize>
__device__ __forceinline__ void widen(float (&f)[16 / kSize], uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (kSize == 4) {
      f[j] = __uint_as_float(w[j]);
    } else {
      f[(2 * j) % (16 / kSize)] = __uint_as_float(w[j] << 16);
      f[(2 * j + 1) % (16 / kSize)] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
}

// Sum of the squares of a thread's part.
template <int kSize>
__device__ __forceinline__ double part_squares(const Part& t) {
  constexpr int kVec = 16 / kSize;
  float most = fabsf(t.one);
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    if (kSize == 2) {  // NaN where all are
      const uint32_t m = absmax_bf16x2(absmax_bf16x2(t.v[j].x, t.v[j].y), absmax_bf16x2(t.v[j].z, t.v[j].w));
      most = fmaxf(most, __uint_as_float(amax_bits_of(m)));
    } else {
      float f[kVec];
      widen<kSize>(f, t.v[j]);
#pragma unroll
      for (int k = 0; k < kVec; ++k) most = fmaxf(most, fabsf(f[k]));
    }
  }
  if (most == 0.0f || (most >= 0x1p-40f && most <= 0x1p60f)) {  // a NaN is dropped by fmaxf
    float sum = t.one * t.one;
#pragma unroll
    for (int j = 0; j < kVecs; j += 8 / kVec) {
      float part = 0.0f;
#pragma unroll
      for (int h = 0; h < 8 / kVec; ++h) {
        float f[kVec];
        widen<kSize>(f, t.v[j + h]);
#pragma unroll
        for (int k = 0; k < kVec; ++k) part = __fmaf_rn(f[k], f[k], part);
      }
      sum += part;
    }
    return sum;
  }
  double sum = static_cast<double>(t.one) * t.one;
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    float f[kVec];
    widen<kSize>(f, t.v[j]);
#pragma unroll
    for (int k = 0; k < kVec; ++k) sum += static_cast<double>(f[k]) * f[k];
  }
  return sum;
}

// The block's sum of v, the same in every thread.
__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) v += red[i];
  return v;
}

template <int kCap>
__global__ void __launch_bounds__(kThreads, 4)
    squares_kernel(const __grid_constant__ Table<kCap> tab, double* partial) {
  __shared__ double red[kWarps];
  grid_wait();
  const int32_t chunks = tab.first[tab.count], step = static_cast<int32_t>(gridDim.x);
  int32_t c = static_cast<int32_t>(blockIdx.x);  // the grid is no larger than the chunks
  Chunk k = chunk_of(tab, c);
  Part t;
  load_part(t, k);
  double sum = 0.0;
  while (true) {
    const int32_t size = k.size;
    const bool more = c < chunks - step;
    Part next = {};
    if (more) {
      c += step;
      k = chunk_of(tab, c);
      load_part(next, k);
    }
    sum += size == 4 ? part_squares<4>(t) : part_squares<2>(t);
    if (!more) break;
    t = next;
  }
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// The norm from the sum of all squares.  What scales the tensors is this fp32 value,
// not the fp64 root: the same norm handed back as a given one has to give the same
// result, zeros past fp32's range among them.
__device__ __forceinline__ float root_of(double sum) { return static_cast<float>(sqrt(sum)); }

// The norm from all partial sums, in one order.
__device__ __forceinline__ float norm_of(const double* partial, int32_t partials, double* red) {
  double sum = 0.0;
  for (int32_t i = threadIdx.x; i < partials; i += kThreads) sum += __ldg(partial + i);
  return root_of(block_sum(sum, red));
}

__global__ void __launch_bounds__(kThreads)
    norm_kernel(const double* partial, int32_t partials, float* norm) {
  __shared__ double red[kWarps];
  grid_wait();
  const float v = norm_of(partial, partials, red);
  if (threadIdx.x == 0) *norm = v;
}

// What the tensors are multiplied by.  Below fp32's normal values a factor would have
// lost bits that the products need not lose (1e38 clipped to 1e-7): there it is
// `wide`, else that is 0.
struct Factor {
  float f;
  double wide;
};

// A NaN is not below the limit: it becomes the factor.
__device__ __forceinline__ Factor factor_of(float norm, float most) {
  if (norm <= most) return {1.0f, 0.0};
  const double q = static_cast<double>(most) / norm;
  return {static_cast<float>(q), q < 0x1p-126 ? q : 0.0};
}

template <bool kWide>
__device__ __forceinline__ float times(float x, const Factor& f) {
  return kWide ? static_cast<float>(x * f.wide) : x * f.f;
}

template <int kSize, bool kWide>
__device__ __forceinline__ uint4 scale_vec(uint4 v, const Factor& f) {
  constexpr int kVec = 16 / kSize;
  float x[kVec];
  widen<kSize>(x, v);
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    w[k] = kSize == 4 ? __float_as_uint(times<kWide>(x[k], f))
                      : bf16x2_of(times<kWide>(x[(2 * k) % kVec], f), times<kWide>(x[(2 * k + 1) % kVec], f));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int kSize, bool kWide>
__device__ __forceinline__ void store_part(const Part& t, const Chunk& k, const Factor& f) {
  uint8_t* const to = k.out + k.head * kSize;
  const bool vectors = (reinterpret_cast<uintptr_t>(to) & 15) == 0;
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int32_t i = threadIdx.x + j * kThreads;
    if (i >= k.vecs) continue;
    const uint4 v = scale_vec<kSize, kWide>(t.v[j], f);
    if (vectors) {
      __stcs(reinterpret_cast<uint4*>(to) + i, v);
    } else {  // the tensor and its output lie differently in their 16 bytes
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 16 / kSize; ++e) {
        if (kSize == 4)
          reinterpret_cast<uint32_t*>(to)[i * 4 + e] = w[e % 4];
        else
          reinterpret_cast<uint16_t*>(to)[i * 8 + e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
      }
    }
  }
  const int32_t at = single_of(k);
  if (at >= 0) store_one(k.out + at, kSize, times<kWide>(t.one, f));
}

__device__ __forceinline__ void scale_part(const Part& t, const Chunk& k, const Factor& f) {
  if (f.wide != 0.0) {
    if (k.size == 4)
      store_part<4, true>(t, k, f);
    else
      store_part<2, true>(t, k, f);
  } else if (k.size == 4) {
    store_part<4, false>(t, k, f);
  } else {
    store_part<2, false>(t, k, f);
  }
}

struct ClipParams {
  const double* partial;
  const float* given;  // the norm, or nullptr: from the partial sums
  float* norm;         // where the first block writes it, or nullptr
  float most;
  int32_t partials;
  bool in_place;       // a factor of 1 writes nothing
};

template <int kCap>
__global__ void __launch_bounds__(kThreads, 4)
    scale_kernel(const __grid_constant__ Table<kCap> tab, const ClipParams p) {
  __shared__ double red[kWarps];
  const int32_t step = static_cast<int32_t>(gridDim.x);
  int32_t c = tab.first[tab.count] - 1 - static_cast<int32_t>(blockIdx.x);  // at least 0
  Chunk k = chunk_of(tab, c);
  grid_wait();
  Part t;
  load_part(t, k);
  const float norm = p.given != nullptr ? __ldg(p.given) : norm_of(p.partial, p.partials, red);
  if (p.norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *p.norm = norm;
  const Factor f = factor_of(norm, p.most);
  if (f.f == 1.0f && p.in_place) return;
  while (true) {
    const Chunk last = k;
    const bool more = c >= step;
    Part next = {};
    if (more) {
      c -= step;
      k = chunk_of(tab, c);
      load_part(next, k);
    }
    scale_part(t, last, f);
    if (!more) break;
    t = next;
  }
}

// Up to kClusterChunks chunks: norm and scaling in one launch, of one cluster
// whose blocks exchange their sums through distributed shared memory, without
// scratch.  (Three tensors of 1000 elements in all: 4.2 us on the GPU instead of
// 6.0, and a launch and an allocation less on the host.)
constexpr int kClusterBlocks = 8, kClusterChunks = 64;

__global__ void __launch_bounds__(kThreads)
    cluster_kernel(const __grid_constant__ Table<kSmall> tab, const ClipParams p, bool write) {
  __shared__ double red[kWarps];
  __shared__ double mine;
  const int32_t chunks = tab.first[tab.count], step = static_cast<int32_t>(gridDim.x);
  const int32_t first = static_cast<int32_t>(blockIdx.x);  // the grid is no larger than the chunks
  grid_wait();
  double sum = 0.0;
  Part t;
  for (int32_t c = first; c < chunks; c += step) {
    const Chunk k = chunk_of(tab, c);
    load_part(t, k);
    sum += k.size == 4 ? part_squares<4>(t) : part_squares<2>(t);
  }
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) mine = sum;
  cluster_arrive();
  cluster_wait();
  double total = 0.0;
  for (int32_t b = 0; b < step; ++b) total += ld_cluster_f64(map_cluster(smem_addr(&mine), b));
  cluster_arrive();  // waited for below: a block's sum is read until then
  const float norm = root_of(total);
  if (first == 0 && threadIdx.x == 0) *p.norm = norm;
  const Factor f = factor_of(norm, p.most);
  if (write && !(f.f == 1.0f && p.in_place)) {
    for (int32_t c = first; c < chunks; c += step) {
      const Chunk k = chunk_of(tab, c);
      if (chunks > step) load_part(t, k);  // else t still holds the only one
      scale_part(t, k, f);
    }
  }
  cluster_wait();
}

// One table after the other is handed to `use`; empty tensors are left out.
template <int kCap, typename F>
gq_status for_tables(const void* const* in, void* const* out, const int64_t* sizes,
                     const int32_t* dtypes, int32_t count, F use) {
  Table<kCap> tab;
  int32_t i = 0;
  while (i < count) {
    tab.count = 0;
    int64_t chunks = 0;
    for (; i < count && tab.count < kCap; ++i) {
      if (sizes[i] == 0) continue;
      const int64_t bytes = sizes[i] * (dtypes[i] == GQ_DTYPE_F32 ? 4 : 2);
      const int64_t more = (bytes + kChunk - 1) / kChunk;
      const int32_t t = tab.count++;
      tab.in[t] = static_cast<const uint8_t*>(in[i]);
      tab.out[t] = static_cast<uint8_t*>(out != nullptr ? out[i] : const_cast<void*>(in[i]));
      tab.size[t] = sizes[i] | (dtypes[i] == GQ_DTYPE_F32 ? kF32Bit : 0);
      tab.first[t] = static_cast<int32_t>(chunks);
      chunks += more;
    }
    if (tab.count == 0) break;
    tab.first[tab.count] = static_cast<int32_t>(chunks);
    const gq_status st = use(tab);
    if (st != GQ_OK) return st;
  }
  return GQ_OK;
}

unsigned grid_of(const DeviceInfo& info, int32_t chunks) {
  const int32_t most = std::min(8 * info.sm_count, kMostBlocks);
  return static_cast<unsigned>(std::min(chunks, most));
}

template <int kCap>
gq_status run(const DeviceInfo& info, const void* const* in, void* const* out, bool write,
              const int64_t* sizes, const int32_t* dtypes, int32_t count, float most,
              const float* given, void* workspace, float* norm, cudaStream_t stream) {
  double* const partial = static_cast<double*>(workspace);
  int32_t partials = 0;
  gq_status st = GQ_OK;
  if (given == nullptr) {
    st = for_tables<kCap>(in, out, sizes, dtypes, count, [&](const Table<kCap>& tab) {
      const unsigned grid = grid_of(info, tab.first[tab.count]);
      double* const to = partial + partials;
      partials += static_cast<int32_t>(grid);
      return launch_chained("grad_norm: launch", squares_kernel<kCap>, dim3(grid), kThreads, 0,
                            stream, 1, tab, to);
    });
    if (st != GQ_OK) return st;
  }
  bool told = false;  // a launch of the scaling writes the norm
  if (write) {
    st = for_tables<kCap>(in, out, sizes, dtypes, count, [&](const Table<kCap>& tab) {
      ClipParams p = {partial, given, told ? nullptr : norm, most, partials, out == nullptr};
      told = true;
      return launch_chained("clip_grads: launch", scale_kernel<kCap>,
                            dim3(grid_of(info, tab.first[tab.count])), kThreads, 0, stream, 1, tab, p);
    });
    if (st != GQ_OK) return st;
  }
  if (norm == nullptr || told) return GQ_OK;
  return launch_chained("grad_norm: launch", norm_kernel, dim3(1), kThreads, 0, stream, 1,
                        static_cast<const double*>(partial), partials, norm);
}

int64_t chunks_of(const int64_t* sizes, const int32_t* dtypes, int32_t count) {
  int64_t chunks = 0;
  for (int32_t i = 0; i < count; ++i)
    chunks += (sizes[i] * (dtypes[i] == GQ_DTYPE_F32 ? 4 : 2) + kChunk - 1) / kChunk;
  return chunks;
}

// Whether one cluster does it.
bool is_small(const int64_t* sizes, const int32_t* dtypes, int32_t count) {
  if (count > kSmall) return false;
  const int64_t chunks = chunks_of(sizes, dtypes, count);
  return chunks > 0 && chunks <= kClusterChunks;
}

struct Range {
  uintptr_t from, to;
};

}  // namespace

// The partial sums of one launch per table.
size_t workspace_bytes(const int64_t* sizes, const int32_t* dtypes, int32_t count) {
  if (is_small(sizes, dtypes, count)) return 0;
  return static_cast<size_t>((count + kLarge - 1) / kLarge) * kMostBlocks * sizeof(double);
}

// Whether an element would be written twice, or written through one pointer
// and read through another: outputs that overlap, an input that overlaps an output
// other than its own, a norm that is read inside an output, or one that is written
// inside any tensor.
gq_status check_overlap(const void* const* in, void* const* out, const int64_t* sizes,
                        const int32_t* dtypes, int32_t count, const float* given,
                        const float* norm) {
  std::unique_ptr<Range[]> r(new (std::nothrow) Range[count > 0 ? count : 1]);
  if (!r) return fail(GQ_ERR_UNSUPPORTED, "gq_clip_grads: no host memory for %d tensors", count);
  int32_t n = 0;
  auto range = [&](const void* p, int32_t i) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Range{a, a + static_cast<uintptr_t>(sizes[i]) * (dtypes[i] == GQ_DTYPE_F32 ? 4 : 2)};
  };
  for (int32_t i = 0; i < count; ++i)
    if (sizes[i] > 0) r[n++] = range(out != nullptr ? out[i] : in[i], i);
  std::sort(r.get(), r.get() + n, [](const Range& a, const Range& b) { return a.from < b.from; });
  for (int32_t i = 1; i < n; ++i)
    if (r[i].from < r[i - 1].to)
      return fail(GQ_ERR_INVALID_ARG, "gq_clip_grads: two outputs overlap");
  auto hits_output = [&](const Range& a) {
    // the first output that ends behind a's start
    const Range* const b = std::upper_bound(
        r.get(), r.get() + n, a.from, [](uintptr_t v, const Range& x) { return v < x.to; });
    return b != r.get() + n && b->from < a.to;
  };
  const float* const value = given != nullptr ? given : norm;
  const Range at = {reinterpret_cast<uintptr_t>(value), reinterpret_cast<uintptr_t>(value + 1)};
  if (hits_output(at)) return fail(GQ_ERR_INVALID_ARG, "gq_clip_grads: the norm overlaps an output");
  if (out == nullptr) return GQ_OK;
  for (int32_t i = 0; i < count; ++i) {
    if (sizes[i] == 0) continue;
    const Range a = range(in[i], i);
    if (given == nullptr && a.from < at.to && at.from < a.to)
      return fail(GQ_ERR_INVALID_ARG, "gq_clip_grads: the norm overlaps tensor %d", i);
    if (in[i] != out[i] && hits_output(a))
      return fail(GQ_ERR_INVALID_ARG, "gq_clip_grads: tensor %d overlaps an output", i);
  }
  return GQ_OK;
}

gq_status launch(const DeviceInfo& info, const void* const* in, void* const* out, bool write,
                 const int64_t* sizes, const int32_t* dtypes, int32_t count, float most,
                 const float* given, void* workspace, float* norm, cudaStream_t stream) {
  if (given == nullptr && is_small(sizes, dtypes, count))
    return for_tables<kSmall>(in, out, sizes, dtypes, count, [&](const Table<kSmall>& tab) {
      const ClipParams p = {nullptr, nullptr, norm, most, 0, out == nullptr};
      const unsigned grid = static_cast<unsigned>(std::min(tab.first[tab.count], kClusterBlocks));
      return launch_chained("grad_norm: launch", cluster_kernel, dim3(grid), kThreads, 0, stream,
                            grid, tab, p, write);
    });
  return count <= kSmall ? run<kSmall>(info, in, out, write, sizes, dtypes, count, most, given,
                                       workspace, norm, stream)
                         : run<kLarge>(info, in, out, write, sizes, dtypes, count, most, given,
                                       workspace, norm, stream);
}

}  // namespace clip
}  // namespace gq
