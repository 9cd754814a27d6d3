// gq_gated.cu -- the backward pass of the gated feed-forward block's activation
// and product, a stream over the rows (its grouped products are in
// gq_grouped_mm.cu).  Formulas in gq_gated.cuh.
#include "gq_gated.cuh"
#include "gq_internal.h"

namespace gq {
namespace gated {

namespace {

constexpr int kBlock = 128;
constexpr int kUnit = 16;                       // columns per lane
constexpr int kUnitsPerBlock = kBlock / kUnit;  // 8 lanes share a block
constexpr int kThreads = 256;

struct BackwardParams {
  const uint8_t* g;
  const uint8_t* pre;
  uint8_t* out;        // may be pre: a lane reads its columns before it writes them
  uint8_t* q;
  float* scales;
  uint32_t blocks;     // 128-blocks of all rows, below 2^31
  uint32_t magic;      // block / nb = block * magic >> shift
  int32_t shift;
  int32_t N, nb;       // columns, 128-blocks per row
  int64_t ld_bytes;    // bytes from one row of g to the next
  Act act;
  bool pow2;
};

// Sixteen consecutive elements as fp32 values, from and to memory.
template <bool kF32>
__device__ __forceinline__ void load_unit(float (&v)[kUnit], const uint8_t* p) {
  const uint4* const s = reinterpret_cast<const uint4*>(p);
#pragma unroll
  for (int i = 0; i < (kF32 ? 4 : 2); ++i) {
    const uint4 x = __ldcs(s + i);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (kF32) {
        v[4 * i + j] = __uint_as_float(w[j]);
      } else {  // a bf16 value is the upper half of its fp32
        v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
        v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    }
  }
}

template <bool kF32>
__device__ __forceinline__ void store_unit(uint8_t* p, const float (&v)[kUnit]) {
  uint4* const d = reinterpret_cast<uint4*>(p);
#pragma unroll
  for (int i = 0; i < (kF32 ? 4 : 2); ++i) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = kF32 ? __float_as_uint(v[4 * i + j]) : bf16x2_of(v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
    d[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Scale of a 1x128 block whose 16-column units eight neighbouring lanes hold;
// a NaN does not count in its amax.
__device__ __forceinline__ float block_scale(const float (&v)[kUnit], bool pow2) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < kUnit; ++i) m = fmaxf(m, fabsf(v[i]));
#pragma unroll
  for (int o = kUnitsPerBlock / 2; o > 0; o >>= 1)
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return scale_from_amax_bits(__float_as_uint(m), pow2);
}

__device__ __forceinline__ uint4 cast_unit(const float (&v)[kUnit], float s) {
  return make_uint4(quant4f(make_float4(v[0], v[1], v[2], v[3]), s),
                    quant4f(make_float4(v[4], v[5], v[6], v[7]), s),
                    quant4f(make_float4(v[8], v[9], v[10], v[11]), s),
                    quant4f(make_float4(v[12], v[13], v[14], v[15]), s));
}

// Eight lanes per 128 columns of a row, of both its halves: read once, the
// gradients formed in fp32 and rounded or quantized from there.  HBM bounds it;
// the logistic function with exp itself costs issue slots (62 %) that are free.
// 16,640 x 4096 bf16 to bf16 and e4m3, 822 MB: 130 us, 6.3 TB/s.
template <bool kF32>
__global__ void __launch_bounds__(kThreads) backward_kernel(const BackwardParams p) {
  grid_wait();
  constexpr int kSize = kF32 ? 4 : 2;
  const int lane = threadIdx.x & 31;
  const uint32_t i = (blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * 4 + (lane >> 3);
  const uint32_t row =
      i < p.blocks ? static_cast<uint32_t>(static_cast<uint64_t>(i) * p.magic >> p.shift) : 0u;
  const int32_t b = static_cast<int32_t>(i - row * static_cast<uint32_t>(p.nb));
  const int32_t col = b * kBlock + (lane & 7) * kUnit;
  // N % 16 == 0: a unit is wholly inside or outside
  const bool in = i < p.blocks && col < p.N;
  const bool lead = i < p.blocks && (lane & 7) == 0;
  const int64_t at = static_cast<int64_t>(row) * 2 * p.N + col;
  float g[kUnit] = {}, x[kUnit] = {}, u[kUnit] = {};
  if (in) {
    load_unit<kF32>(g, p.g + row * p.ld_bytes + static_cast<int64_t>(col) * kSize);
    load_unit<kF32>(x, p.pre + at * kSize);
    load_unit<kF32>(u, p.pre + (at + p.N) * kSize);
  }
#pragma unroll
  for (int j = 0; j < kUnit; ++j) {
    const float s = sigma(act_z(p.act, x[j]));
    // the slope first: where it is 0, g u may be past fp32's range
    const float dx = g[j] * act_slope(p.act, x[j], s) * u[j];
    u[j] = g[j] * act_value(x[j], s);
    x[j] = dx;
  }
  if (p.out != nullptr && in) {
    store_unit<kF32>(p.out + at * kSize, x);
    store_unit<kF32>(p.out + (at + p.N) * kSize, u);
  }
  if (p.q == nullptr) return;
  const float sx = block_scale(x, p.pow2), su = block_scale(u, p.pow2);
  if (in) {
    *reinterpret_cast<uint4*>(p.q + at) = cast_unit(x, sx);
    *reinterpret_cast<uint4*>(p.q + at + p.N) = cast_unit(u, su);
  }
  if (lead) {
    float* const d = p.scales + static_cast<int64_t>(row) * 2 * p.nb + b;
    d[0] = sx;
    d[p.nb] = su;
  }
}

}  // namespace

gq_status launch_backward(const void* g, const void* pre, bool f32, int64_t rows, int64_t N,
                          int64_t ld, int activation, void* out, void* q, float* scales, bool pow2,
                          cudaStream_t stream) {
  BackwardParams p;
  p.g = static_cast<const uint8_t*>(g);
  p.pre = static_cast<const uint8_t*>(pre);
  p.out = static_cast<uint8_t*>(out);
  p.q = static_cast<uint8_t*>(q);
  p.scales = scales;
  p.N = static_cast<int32_t>(N);
  p.nb = static_cast<int32_t>((N + kBlock - 1) / kBlock);
  p.ld_bytes = ld * (f32 ? 4 : 2);
  const int64_t blocks = rows * p.nb;
  if (blocks > INT32_MAX)
    return fail(GQ_ERR_UNSUPPORTED, "gated_backward: %lld blocks of 128",
                static_cast<long long>(blocks));
  p.blocks = static_cast<uint32_t>(blocks);
  // exact for blocks below 2^31, as in moe_sort
  int l = 0;
  while ((1 << l) < p.nb) ++l;
  p.shift = 31 + l;
  p.magic = static_cast<uint32_t>(((uint64_t(1) << p.shift) + p.nb - 1) / p.nb);
  p.act = act_of(activation);
  p.pow2 = pow2;
  constexpr int kPer = kThreads / 32 * 4;  // 128-blocks per thread block
  const int64_t grid = (blocks + kPer - 1) / kPer;
  return launch_chained("gated_backward: launch", f32 ? backward_kernel<true> : backward_kernel<false>,
                        dim3(static_cast<unsigned>(grid)), kThreads, 0, stream, 1, p);
}

}  // namespace gated
}  // namespace gq
