// gq_grouped_mm.cu -- the grouped product of block-quantized rows with
// block-quantized stacked weights, one expert per token group:
//   forward     out[m][n] = sum_k A[m][k] * W[e][n][k]
//   transposed  out[m][k] = sum_n A[m][n] * W[e][n][k]
// with A = qa / sa (one scale per row and 128 contraction columns) and
// W = qb / sb (one scale per 128x128 block).  Within a 128-block of the
// contraction both scales are constant for an output row and 128 output
// columns, so each block's e4m3 products are summed plain in fp32 and the
// sum enters the fp32 accumulator once, times 1/sa * 1/sb.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gq_device.cuh"
#include "gq_internal.h"

namespace gq {
namespace gmm {

constexpr int kBlock = 128;
constexpr int kT = 64;       // rows and columns of a tile
constexpr int kStep = 32;    // contraction columns per shared-memory step
constexpr int kThreads = 256;

struct Params {
  const uint8_t* qa;
  const float* sa;
  const uint8_t* qb;
  const float* sb;
  const int32_t* offs;
  uint16_t* out;
  int64_t M;
  int32_t E, inner, outer;  // contraction extent, output columns
  int32_t N, K;
};

__device__ __forceinline__ float e4m3_value(uint8_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(b)));
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu)));
}

// One block per 64x64 output tile of a group; 4x4 outputs per thread.
template <bool kTransposed>
__global__ void __launch_bounds__(kThreads) simple_kernel(const Params p) {
  __shared__ int32_t ends[kMaxGroups];
  __shared__ float as[kStep][kT + 1];
  __shared__ float bs[kStep][kT + 1];
  if (threadIdx.x < 32)
    build_ends(p.offs, 0, p.E, static_cast<int32_t>(p.M), ends, threadIdx.x);
  __syncthreads();
  int32_t left = blockIdx.x, g = 0, m0 = 0, m1 = 0;
  for (;; ++g) {
    if (g == p.E) return;
    m0 = g > 0 ? ends[g - 1] : 0;
    m1 = ends[g];
    const int32_t n = (m1 - m0 + kT - 1) / kT;
    if (left < n) break;
    left -= n;
  }
  m0 += left * kT;
  const int32_t c0 = blockIdx.y * kT;
  const int32_t nb_in = (p.inner + kBlock - 1) / kBlock, nb_k = (p.K + kBlock - 1) / kBlock;
  const int32_t nb_n = (p.N + kBlock - 1) / kBlock;
  const uint8_t* w = p.qb + static_cast<int64_t>(g) * p.N * p.K;
  const float* sbg = p.sb + static_cast<int64_t>(g) * nb_n * nb_k;
  const int tr = threadIdx.x / 16, tc = threadIdx.x % 16;
  float acc[4][4] = {};
  for (int32_t kb = 0; kb < nb_in; ++kb) {
    float sum[4][4] = {};
    for (int32_t k0 = kb * kBlock; k0 < min((kb + 1) * kBlock, p.inner); k0 += kStep) {
      for (int i = threadIdx.x; i < kT * kStep; i += kThreads) {
        const int32_t k = i % kStep, r = i / kStep;
        const bool in = m0 + r < m1 && k0 + k < p.inner;
        as[k][r] = in ? e4m3_value(p.qa[static_cast<int64_t>(m0 + r) * p.inner + k0 + k]) : 0.0f;
      }
      for (int i = threadIdx.x; i < kT * kStep; i += kThreads) {
        const int32_t k = kTransposed ? i / kT : i % kStep;
        const int32_t c = kTransposed ? i % kT : i / kStep;
        const bool in = c0 + c < p.outer && k0 + k < p.inner;
        const int64_t at = kTransposed ? static_cast<int64_t>(k0 + k) * p.K + c0 + c
                                       : static_cast<int64_t>(c0 + c) * p.K + k0 + k;
        bs[k][c] = in ? e4m3_value(w[at]) : 0.0f;
      }
      __syncthreads();
      for (int k = 0; k < kStep; ++k) {
        float a[4], b[4];
        for (int i = 0; i < 4; ++i) {
          a[i] = as[k][tr * 4 + i];
          b[i] = bs[k][tc * 4 + i];
        }
        for (int i = 0; i < 4; ++i)
          for (int j = 0; j < 4; ++j) sum[i][j] = __fmaf_rn(a[i], b[j], sum[i][j]);
      }
      __syncthreads();
    }
    const int32_t cb = c0 / kBlock;
    const float rb = __frcp_rn(kTransposed ? sbg[kb * nb_k + cb] : sbg[cb * nb_k + kb]);
    for (int i = 0; i < 4; ++i) {
      const int32_t m = m0 + tr * 4 + i;
      if (m >= m1) continue;
      const float r = __fmul_rn(__frcp_rn(p.sa[static_cast<int64_t>(m) * nb_in + kb]), rb);
      for (int j = 0; j < 4; ++j) acc[i][j] = __fmaf_rn(sum[i][j], r, acc[i][j]);
    }
  }
  for (int i = 0; i < 4; ++i) {
    const int32_t m = m0 + tr * 4 + i;
    for (int j = 0; j < 4; ++j) {
      const int32_t c = c0 + tc * 4 + j;
      if (m < m1 && c < p.outer)
        p.out[static_cast<int64_t>(m) * p.outer + c] =
            __bfloat16_as_ushort(__float2bfloat16_rn(acc[i][j]));
    }
  }
}

gq_status setup(DeviceInfo& info) {
  (void)info;
  return GQ_OK;
}

gq_status launch(const DeviceInfo& info, const DebugKnobs& dbg, const void* qa, const float* sa,
                 int64_t M, const void* qb, const float* sb, int32_t N, int32_t K, bool transposed,
                 const int32_t* offs, int32_t E, void* out, cudaStream_t stream) {
  (void)info;
  (void)dbg;
  Params p;
  p.qa = static_cast<const uint8_t*>(qa);
  p.sa = sa;
  p.qb = static_cast<const uint8_t*>(qb);
  p.sb = sb;
  p.offs = offs;
  p.out = static_cast<uint16_t*>(out);
  p.M = M;
  p.E = E;
  p.N = N;
  p.K = K;
  p.inner = transposed ? N : K;
  p.outer = transposed ? K : N;
  const int64_t mt = M / kT + (E < M ? E : M);  // at least the row tiles of any offsets
  const dim3 grid(static_cast<unsigned>(mt), (p.outer + kT - 1) / kT);
  if (transposed)
    simple_kernel<true><<<grid, kThreads, 0, stream>>>(p);
  else
    simple_kernel<false><<<grid, kThreads, 0, stream>>>(p);
  return check_cuda(cudaGetLastError(), "grouped_mm: launch");
}

}  // namespace gmm
}  // namespace gq
