// gq_block.cu -- e4m3 quantization with one fp32 scale per block of 128:
// rows cut into 1x128 blocks (activations, gradients), optionally written to
// the expert-sorted rows of each token, and stacked weights (E, N, K) cut
// into 128x128 tiles.  For a block b
//     amax  = max |x| over b
//     scale = 448 / max(amax, 1e-12)            IEEE fp32 division
//     q     = e4m3(fp32(x * scale))             RNE, saturating to +-448
// (the scale rounded down to a power of two with GQ_SCALE_POW2), the same
// scale and cast as the per-group kernels.  The amax is a maximum and the
// scale and product are fp32: nothing is rounded below 32 bits before the
// cast.  Both kernels are bound by HBM: 2 (4) bytes read and 1 written per
// element.
//
// The unit of work is 16 consecutive columns (K is a multiple of 16): one
// lane reads a unit's 32 (bf16) or 64 (fp32) bytes and stores its 16 output
// bytes at once, and eight lanes hold one 128-column block.
#include "gq_device.cuh"
#include "gq_internal.h"

namespace gq {
namespace block {

constexpr int kBlock = 128;
constexpr int kUnit = 16;                    // columns per lane
constexpr int kUnitsPerBlock = kBlock / kUnit;  // 8 lanes share a block
constexpr int kThreads = 256;

// Sixteen consecutive elements in registers.
template <bool kF32>
struct Unit;

template <>
struct Unit<false> {
  static constexpr int kBytes = 2 * kUnit;
  uint4 v[2];
  __device__ __forceinline__ void load(const uint8_t* p) {
    v[0] = __ldcs(reinterpret_cast<const uint4*>(p));
    v[1] = __ldcs(reinterpret_cast<const uint4*>(p) + 1);
  }
  __device__ __forceinline__ void clear() { v[0] = v[1] = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ uint32_t amax_bits() const {
    const uint32_t a = absmax_bf16x2(absmax_bf16x2(v[0].x, v[0].y), absmax_bf16x2(v[0].z, v[0].w));
    const uint32_t b = absmax_bf16x2(absmax_bf16x2(v[1].x, v[1].y), absmax_bf16x2(v[1].z, v[1].w));
    // the last maximum, with zero, drops a NaN that all values of a half share;
    // its bits would win every comparison that follows
    return amax_bits_of(absmax_bf16x2(absmax_bf16x2(a, b), 0u));
  }
  __device__ __forceinline__ uint4 cast(float s) const {
    return make_uint4(quant4(v[0].x, v[0].y, s, s, s, s), quant4(v[0].z, v[0].w, s, s, s, s),
                      quant4(v[1].x, v[1].y, s, s, s, s), quant4(v[1].z, v[1].w, s, s, s, s));
  }
};

template <>
struct Unit<true> {
  static constexpr int kBytes = 4 * kUnit;
  float4 v[4];
  __device__ __forceinline__ void load(const uint8_t* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __ldcs(reinterpret_cast<const float4*>(p) + i);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  __device__ __forceinline__ uint32_t amax_bits() const {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m = fmaxf(m, fmaxf(fmaxf(fabsf(v[i].x), fabsf(v[i].y)), fmaxf(fabsf(v[i].z), fabsf(v[i].w))));
    return __float_as_uint(m);
  }
  __device__ __forceinline__ uint4 cast(float s) const {
    return make_uint4(quant4f(v[0], s), quant4f(v[1], s), quant4f(v[2], s), quant4f(v[3], s));
  }
};

struct RowParams {
  const uint8_t* x;
  uint8_t* q;
  float* scales;
  const int32_t* pos;  // (rows, top_k) destination rows, or nullptr: row r goes to row r
  uint32_t blocks;     // 128-blocks of all rows, below 2^31
  uint32_t out_rows;   // of pos
  int64_t ld_bytes;    // bytes from one input row to the next
  int32_t K, nb;       // columns, 128-blocks per row
  uint32_t magic;      // block / nb = block * magic >> shift
  int32_t shift;
  int32_t top_k;
  bool pow2;
};

// Eight lanes per 1x128 block, four consecutive blocks (of one row or of
// several) per warp; a block's values and its token's positions are loaded at
// the same time.  A token is read once and its quantized block stored to each
// of its sorted rows.  65,536 x 4096 bf16: 115 us, 7.1 TB/s; to one sorted row
// each 120 us; 32,768 x 4096 to six rows each 164 us, 6.7 TB/s; 32,768 x 4096 fp32
// 95 us, 7.1 TB/s.  Issue slots
// are the next limit: with a division for the row and 64-bit positions 126, 146
// and 163 us.  (Two blocks per lane group and positions before values, to skip
// tokens without a live slot, were slower.)
constexpr int kPosBatch = 8;  // positions held in registers

template <bool kF32, bool kStream>
__global__ void __launch_bounds__(kThreads) rows_kernel(const RowParams p) {
  grid_wait();
  const int lane = threadIdx.x & 31;
  const uint32_t i = (blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * 4 + (lane >> 3);
  const uint32_t row =
      i < p.blocks ? static_cast<uint32_t>(static_cast<uint64_t>(i) * p.magic >> p.shift) : 0u;
  const int32_t b = static_cast<int32_t>(i - row * static_cast<uint32_t>(p.nb));
  const int32_t col = b * kBlock + (lane & 7) * kUnit;
  // K % 16 == 0: a unit is wholly inside or outside
  const bool in = i < p.blocks && col < p.K;
  const bool lead = i < p.blocks && (lane & 7) == 0;
  Unit<kF32> u;
  if (in)
    u.load(p.x + row * p.ld_bytes + static_cast<int64_t>(col) * (kF32 ? 4 : 2));
  else
    u.clear();
  const int32_t* pos = p.pos + static_cast<int64_t>(row) * p.top_k;
  int32_t to[kPosBatch];  // the first destination rows, -1 for dropped slots
  if (p.pos != nullptr) {
#pragma unroll
    for (int j = 0; j < kPosBatch; ++j) to[j] = j < p.top_k ? __ldg(pos + j) : -1;
  }
  uint32_t m = u.amax_bits();
#pragma unroll
  for (int o = kUnitsPerBlock / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float s = scale_from_amax_bits(m, p.pow2);
  const uint4 q = u.cast(s);
  uint8_t* const q0 = p.q + col;
  float* const s0 = p.scales + b;
  auto store = [&](int32_t r) {
    uint4* const to_q = reinterpret_cast<uint4*>(q0 + static_cast<int64_t>(r) * p.K);
    if (in && kStream) __stcs(to_q, q);
    if (in && !kStream) *to_q = q;
    if (lead) s0[static_cast<int64_t>(r) * p.nb] = s;
  };
  if (p.pos == nullptr) {
    store(static_cast<int32_t>(row));
    return;
  }
  // a negative position is past every row as an unsigned number
#pragma unroll
  for (int j = 0; j < kPosBatch; ++j)
    if (static_cast<uint32_t>(to[j]) < p.out_rows) store(to[j]);
  for (int32_t j = kPosBatch; j < p.top_k; ++j) {
    const int32_t r = __ldg(pos + j);
    if (static_cast<uint32_t>(r) < p.out_rows) store(r);
  }
}

// An output of this size or more leaves L2 anyway before it is read: stored
// past it (8192 tokens of 4096 columns to eight rows: 52.3 us instead of 53.9;
// 16,384 rows of 2048 columns, which stay in L2: 7.2 us instead of 6.5).
constexpr int64_t kStreamBytes = int64_t(128) << 20;

struct TileParams {
  const uint8_t* w;
  uint8_t* q;
  float* scales;
  int32_t N, K, nn, nk;  // sizes of one matrix, tiles along each
  bool pow2;
};

constexpr int kTileUnits = kBlock * kUnitsPerBlock / kThreads;  // 4 units per thread

// One block of 256 threads per 128x128 tile, held in registers between the
// amax and the cast: thread t owns unit t % 8 of rows t / 8 + 32 i.  16 x 8192
// x 4096 bf16: 224 us, 7.2 TB/s.
template <bool kF32>
__global__ void __launch_bounds__(kThreads) tiles_kernel(const TileParams p) {
  __shared__ uint32_t red[kThreads / 32];
  grid_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t per = static_cast<int64_t>(p.nn) * p.nk;
  const int64_t e = blockIdx.x / per;
  const int32_t r = static_cast<int32_t>(blockIdx.x % per);
  const int32_t n0 = (r / p.nk) * kBlock + (threadIdx.x >> 3);
  const int32_t col = (r % p.nk) * kBlock + (threadIdx.x & 7) * kUnit;
  const int64_t at = (e * p.N + n0) * p.K + col;
  Unit<kF32> u[kTileUnits];
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < kTileUnits; ++i) {
    if (col < p.K && n0 + 32 * i < p.N)
      u[i].load(p.w + (at + static_cast<int64_t>(32 * i) * p.K) * (kF32 ? 4 : 2));
    else
      u[i].clear();
  }
#pragma unroll
  for (int i = 0; i < kTileUnits; ++i) m = max(m, u[i].amax_bits());
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red[warp] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) m = max(m, red[i]);
  const float s = scale_from_amax_bits(m, p.pow2);
  if (threadIdx.x == 0) p.scales[blockIdx.x] = s;
#pragma unroll
  for (int i = 0; i < kTileUnits; ++i)
    if (col < p.K && n0 + 32 * i < p.N)
      __stcs(reinterpret_cast<uint4*>(p.q + at + static_cast<int64_t>(32 * i) * p.K), u[i].cast(s));
}

gq_status launch_rows(const void* x, bool f32, int64_t rows, int64_t K,
                      int64_t ld, const int32_t* pos, int32_t top_k, int64_t out_rows, void* out,
                      float* scales, bool pow2, cudaStream_t stream) {
  RowParams p;
  p.x = static_cast<const uint8_t*>(x);
  p.q = static_cast<uint8_t*>(out);
  p.scales = scales;
  p.pos = pos;
  constexpr int64_t kMaxRows = int64_t(1) << 31;  // positions are int32
  p.out_rows = static_cast<uint32_t>(out_rows < kMaxRows ? out_rows : kMaxRows);
  p.ld_bytes = ld * (f32 ? 4 : 2);
  p.K = static_cast<int32_t>(K);
  p.nb = static_cast<int32_t>((K + kBlock - 1) / kBlock);
  const int64_t blocks = rows * p.nb;
  if (blocks > INT32_MAX)
    return fail(GQ_ERR_UNSUPPORTED, "block_rows: %lld blocks of 128", static_cast<long long>(blocks));
  p.blocks = static_cast<uint32_t>(blocks);
  // exact for blocks below 2^31, as in moe_sort
  int l = 0;
  while ((1 << l) < p.nb) ++l;
  p.shift = 31 + l;
  p.magic = static_cast<uint32_t>(((uint64_t(1) << p.shift) + p.nb - 1) / p.nb);
  p.top_k = top_k;
  p.pow2 = pow2;
  constexpr int kPer = kThreads / 32 * 4;  // 128-blocks per thread block
  const int64_t grid = (blocks + kPer - 1) / kPer;
  const bool past_l2 = (pos != nullptr ? static_cast<int64_t>(p.out_rows) : rows) * K >= kStreamBytes;
  void (*kernel)(RowParams) =
      f32 ? (past_l2 ? rows_kernel<true, true> : rows_kernel<true, false>)
          : (past_l2 ? rows_kernel<false, true> : rows_kernel<false, false>);
  return launch_chained("block_rows: launch", kernel, dim3(static_cast<unsigned>(grid)), kThreads, 0,
                        stream, 1, p);
}

gq_status launch_tiles(const void* w, bool f32, int64_t E, int64_t N, int64_t K, void* out,
                       float* scales, bool pow2, cudaStream_t stream) {
  TileParams p;
  p.w = static_cast<const uint8_t*>(w);
  p.q = static_cast<uint8_t*>(out);
  p.scales = scales;
  p.N = static_cast<int32_t>(N);
  p.K = static_cast<int32_t>(K);
  p.nn = static_cast<int32_t>((N + kBlock - 1) / kBlock);
  p.nk = static_cast<int32_t>((K + kBlock - 1) / kBlock);
  p.pow2 = pow2;
  const int64_t tiles = E * p.nn * p.nk;  // the caller keeps it below 2^31
  return launch_chained("block_tiles: launch", f32 ? tiles_kernel<true> : tiles_kernel<false>,
                        dim3(static_cast<unsigned>(tiles)), kThreads, 0, stream, 1, p);
}

}  // namespace block
}  // namespace gq
