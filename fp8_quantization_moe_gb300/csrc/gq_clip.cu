// gq_clip.cu -- the norm over all elements of a list of tensors, and the
// tensors scaled to a largest norm:
//     norm = sqrt(sum of x^2),   y = x * min(1, max_norm / norm)
// Both are streams bound by HBM: the norm reads every element once, the
// scaling reads and writes every element once more.
//
// The tensors are cut into chunks of kChunk elements; a block takes a
// contiguous range of the chunks of all tensors and walks the table of
// tensors, which comes with the launch's parameters: nothing is copied to the
// device beforehand, so a call can be captured.
//
// A thread sums the squares of up to 32 elements in fp32, eight to a partial
// sum, and everything beyond that in fp64 (one fp64 addition for 32
// elements), in an order that depends on the sizes alone: the result is the
// same in every run.  Squares of values past 2^60, or all below 2^-40, would
// leave fp32's range: such a thread squares in fp64.
#include <algorithm>
#include <memory>
#include <new>

#include "gq_tcgen05.cuh"
#include "gq_internal.h"

namespace gq {
namespace clip {

namespace {

constexpr int kThreads = 256;
constexpr int kPer = 32;                     // elements per thread and chunk
constexpr int kChunk = kThreads * kPer;
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

// The chunks of one block, and the tensor of the current one.
template <int kCap>
struct Walk {
  int32_t t = 0;
  // the tensor of chunk c
  __device__ __forceinline__ void find(const Table<kCap>& tab, int32_t c) {
    int32_t lo = 0, hi = tab.count - 1;  // the last tensor whose first chunk is at or before c
    while (lo < hi) {
      const int32_t mid = (lo + hi + 1) >> 1;
      if (tab.first[mid] <= c)
        lo = mid;
      else
        hi = mid - 1;
    }
    t = lo;
  }
};

// A chunk's elements: `head` single ones up to the first 16-byte boundary,
// `vecs` 16-byte vectors, `tail` single ones behind them.
struct Span {
  int32_t head, vecs, tail;
};

template <int kSize>
__device__ __forceinline__ Span span_of(const uint8_t* p, int32_t n) {
  constexpr int kVec = 16 / kSize;
  Span s;
  s.head = min(n, static_cast<int32_t>((-reinterpret_cast<uintptr_t>(p) & 15) / kSize));
  s.vecs = (n - s.head) / kVec;
  s.tail = n - s.head - s.vecs * kVec;
  return s;
}

template <int kSize>
__device__ __forceinline__ float load_one(const uint8_t* p) {
  return kSize == 4 ? *reinterpret_cast<const float*>(p)
                    : __uint_as_float(uint32_t(*reinterpret_cast<const uint16_t*>(p)) << 16);
}

template <int kSize>
__device__ __forceinline__ void store_one(uint8_t* p, float v) {
  if (kSize == 4)
    *reinterpret_cast<float*>(p) = v;
  else
    *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(bf16x2_of(v, 0.0f) & 0xFFFFu);
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

// Sum of the squares of this thread's elements of a chunk.
template <int kSize>
__device__ __forceinline__ double chunk_squares(const uint8_t* p, int32_t n) {
  constexpr int kVec = 16 / kSize, kVecs = kPer / kVec;
  const Span s = span_of<kSize>(p, n);
  const uint4* const q = reinterpret_cast<const uint4*>(p + s.head * kSize);
  uint4 v[kVecs];
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int32_t i = threadIdx.x + j * kThreads;
    v[j] = i < s.vecs ? __ldg(q + i) : make_uint4(0u, 0u, 0u, 0u);
  }
  // at most 7 + 7 single elements, two warps
  float one = 0.0f;
  const int32_t lane = threadIdx.x & 31;
  if (threadIdx.x < 32 && lane < s.head) one = load_one<kSize>(p + lane * kSize);
  if (threadIdx.x >= 32 && threadIdx.x < 64 && lane < s.tail)
    one = load_one<kSize>(p + (s.head + s.vecs * kVec + lane) * kSize);
  float most = fabsf(one);
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    float f[kVec];
    widen<kSize>(f, v[j]);
#pragma unroll
    for (int k = 0; k < kVec; ++k) most = fmaxf(most, fabsf(f[k]));
  }
  if (most == 0.0f || (most >= 0x1p-40f && most <= 0x1p60f)) {  // a NaN is dropped by fmaxf
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < kVecs; j += 8 / kVec) {
      float part = j == 0 ? one * one : 0.0f;
#pragma unroll
      for (int h = 0; h < 8 / kVec; ++h) {
        float f[kVec];
        widen<kSize>(f, v[j + h]);
#pragma unroll
        for (int k = 0; k < kVec; ++k) part = __fmaf_rn(f[k], f[k], part);
      }
      sum += part;
    }
    return sum;
  }
  double sum = static_cast<double>(one) * one;
#pragma unroll 1
  for (int j = 0; j < kVecs; ++j) {
    float f[kVec];
    widen<kSize>(f, v[j]);
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

// This block's range of the chunks.
__device__ __forceinline__ void my_range(int32_t chunks, int32_t& from, int32_t& to) {
  from = static_cast<int32_t>(static_cast<int64_t>(chunks) * blockIdx.x / gridDim.x);
  to = static_cast<int32_t>(static_cast<int64_t>(chunks) * (blockIdx.x + 1) / gridDim.x);
}

template <int kCap>
__global__ void __launch_bounds__(kThreads)
    squares_kernel(const __grid_constant__ Table<kCap> tab, double* partial) {
  __shared__ double red[kWarps];
  grid_wait();
  int32_t from, to;
  my_range(tab.first[tab.count], from, to);
  Walk<kCap> w;
  w.find(tab, from);
  double sum = 0.0;
  for (int32_t c = from; c < to; ++c) {
    while (tab.first[w.t + 1] <= c) ++w.t;
    const bool f32 = (tab.size[w.t] & kF32Bit) != 0;
    const int64_t e = static_cast<int64_t>(c - tab.first[w.t]) * kChunk;
    const int64_t left = (tab.size[w.t] & ~kF32Bit) - e;
    const int32_t n = left < kChunk ? static_cast<int32_t>(left) : kChunk;
    sum += f32 ? chunk_squares<4>(tab.in[w.t] + e * 4, n) : chunk_squares<2>(tab.in[w.t] + e * 2, n);
  }
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// The norm from all partial sums, in one order.
__device__ __forceinline__ double norm_of(const double* partial, int32_t partials, double* red) {
  double sum = 0.0;
  for (int32_t i = threadIdx.x; i < partials; i += kThreads) sum += __ldg(partial + i);
  return sqrt(block_sum(sum, red));
}

__global__ void __launch_bounds__(kThreads)
    norm_kernel(const double* partial, int32_t partials, float* norm) {
  __shared__ double red[kWarps];
  grid_wait();
  const double v = norm_of(partial, partials, red);
  if (threadIdx.x == 0) *norm = static_cast<float>(v);
}

template <int kSize>
__device__ __forceinline__ void scale_chunk(const uint8_t* p, uint8_t* o, int32_t n, float f) {
  constexpr int kVec = 16 / kSize, kVecs = kPer / kVec;
  if (((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15) != 0) {
    // no vector of the one is a vector of the other
    for (int32_t i = threadIdx.x; i < n; i += kThreads)
      store_one<kSize>(o + i * kSize, load_one<kSize>(p + i * kSize) * f);
    return;
  }
  const Span s = span_of<kSize>(p, n);
  const uint4* const q = reinterpret_cast<const uint4*>(p + s.head * kSize);
  uint4* const d = reinterpret_cast<uint4*>(o + s.head * kSize);
  uint4 v[kVecs];
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int32_t i = threadIdx.x + j * kThreads;
    if (i < s.vecs) v[j] = q[i];
  }
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int32_t i = threadIdx.x + j * kThreads;
    if (i >= s.vecs) continue;
    float x[kVec];
    widen<kSize>(x, v[j]);
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = kSize == 4 ? __float_as_uint(x[k] * f)
                        : bf16x2_of(x[(2 * k) % kVec] * f, x[(2 * k + 1) % kVec] * f);
    d[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  const int32_t lane = threadIdx.x & 31;
  int32_t at = -1;
  if (threadIdx.x < 32 && lane < s.head) at = lane;
  if (threadIdx.x >= 32 && threadIdx.x < 64 && lane < s.tail) at = s.head + s.vecs * kVec + lane;
  if (at >= 0) store_one<kSize>(o + at * kSize, load_one<kSize>(p + at * kSize) * f);
}

struct ClipParams {
  const double* partial;
  const float* given;  // the norm, or nullptr: from the partial sums
  float* norm;         // where the first block writes it, or nullptr
  float most;
  int32_t partials;
};

template <int kCap>
__global__ void __launch_bounds__(kThreads)
    scale_kernel(const __grid_constant__ Table<kCap> tab, const ClipParams p) {
  __shared__ double red[kWarps];
  grid_wait();
  const double norm = p.given != nullptr ? static_cast<double>(__ldg(p.given))
                                         : norm_of(p.partial, p.partials, red);
  if (p.norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *p.norm = static_cast<float>(norm);
  // a NaN is not below the limit: it becomes the factor
  const float f = norm <= p.most ? 1.0f : static_cast<float>(p.most / norm);
  int32_t from, to;
  my_range(tab.first[tab.count], from, to);
  Walk<kCap> w;
  w.find(tab, from);
  for (int32_t c = from; c < to; ++c) {
    while (tab.first[w.t + 1] <= c) ++w.t;
    const uint8_t* in = tab.in[w.t];
    uint8_t* out = tab.out[w.t];
    if (f == 1.0f && in == out) continue;
    const bool f32 = (tab.size[w.t] & kF32Bit) != 0;
    const int64_t e = static_cast<int64_t>(c - tab.first[w.t]) * kChunk;
    const int64_t left = (tab.size[w.t] & ~kF32Bit) - e;
    const int32_t n = left < kChunk ? static_cast<int32_t>(left) : kChunk;
    if (f32)
      scale_chunk<4>(in + e * 4, out + e * 4, n, f);
    else
      scale_chunk<2>(in + e * 2, out + e * 2, n, f);
  }
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
      const int64_t more = (sizes[i] + kChunk - 1) / kChunk;
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
      ClipParams p = {partial, given, told ? nullptr : norm, most, partials};
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

struct Range {
  uintptr_t from, to;
};

}  // namespace

// The partial sums of one launch per table.
size_t workspace_bytes(int32_t count) {
  return static_cast<size_t>((count + kLarge - 1) / kLarge) * kMostBlocks * sizeof(double);
}

// Whether an element would be written twice, or written through one pointer
// and read through another: outputs that overlap, or an input that overlaps
// an output other than its own.
gq_status check_overlap(const void* const* in, void* const* out, const int64_t* sizes,
                        const int32_t* dtypes, int32_t count) {
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
  if (out == nullptr) return GQ_OK;
  for (int32_t i = 0; i < count; ++i) {
    if (sizes[i] == 0 || in[i] == out[i]) continue;
    const Range a = range(in[i], i);
    // the first output that ends behind a's start
    const Range* const b = std::upper_bound(
        r.get(), r.get() + n, a.from, [](uintptr_t v, const Range& x) { return v < x.to; });
    if (b != r.get() + n && b->from < a.to)
      return fail(GQ_ERR_INVALID_ARG, "gq_clip_grads: tensor %d overlaps an output", i);
  }
  return GQ_OK;
}

gq_status launch(const DeviceInfo& info, const void* const* in, void* const* out, bool write,
                 const int64_t* sizes, const int32_t* dtypes, int32_t count, float most,
                 const float* given, void* workspace, float* norm, cudaStream_t stream) {
  return count <= kSmall ? run<kSmall>(info, in, out, write, sizes, dtypes, count, most, given,
                                       workspace, norm, stream)
                         : run<kLarge>(info, in, out, write, sizes, dtypes, count, most, given,
                                       workspace, norm, stream);
}

}  // namespace clip
}  // namespace gq
