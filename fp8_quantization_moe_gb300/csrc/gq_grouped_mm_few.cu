// gq_grouped_mm_few.cu -- the grouped block-scaled product where the groups
// have few rows (decoding): every touched expert's weights are read once for
// a handful of rows, so HBM bounds it, 1 byte per weight.  512 rows of 64
// experts, K 2064 to N 2832: 59 us, 6.4 TB/s; eight rows of eight experts, K
// 2048 to N 4096: 14.3 us, of which 9.9 us are the weights and most of the
// rest the launch, the first loads and the last tile.
//
// Here the weights are the MMA's M operand (128 output columns) and the rows
// its N operand, up to 128 of them in steps of 16: an MMA costs as many cycles
// as there are rows, and four accumulators keep the tensor cores, the epilogue
// and 96 KB of weights per SM in flight at once.  A lane of the epilogue owns
// an output column and needs every row's factor 1/sa * 1/sb; with few rows
// those shared loads are cheap.
//
// One persistent block per SM; its warps:
//   0-7   epilogue: TMEM lane quarter w % 4 (32 output columns), rows
//         64 (w / 4) and on;
//   8     TMA loads (one lane);
//   9     TMEM allocation and the MMAs (one lane);
//   10    the factors, four 128-blocks at a time, into a ring.
// Every wait is bounded, as in the other kernels.
#include <cuda_bf16.h>

#include "gq_grouped_mm.cuh"
#include "gq_tcgen05.cuh"

namespace gq {
namespace gmm {
namespace {

constexpr int kCols = 128;     // output columns of a tile (the MMA's M)
constexpr int kTok = 128;      // rows of a tile, at most (the MMA's N)
constexpr int kUnit = 16;      // rows of a tile come in units
constexpr int kWarpTok = 64;   // rows of an epilogue warp, at most
constexpr int kWBytes = kCols * kBlock;   // 16 KB
constexpr int kScaleKb = 4;    // 128-blocks per entry of the factor ring
constexpr int kScaleRing = 4;
constexpr int kStages = 6;
constexpr int kStageBytes = kWBytes + kTok * kBlock;
constexpr int kBufs = 512 / kTok;
constexpr int kEpiWarps = 4 * (kTok / kWarpTok);
constexpr int kThreads = (kEpiWarps + 3) * 32;

struct Smem {
  uint8_t stage[kStages][kStageBytes];
  alignas(16) float factor[kScaleRing][kScaleKb][kTok];
  TileTable tiles;
  uint64_t full[kStages];
  uint64_t done[kStages];
  uint64_t acc_empty[kBufs];
  uint64_t fac_full[kScaleRing];
  uint64_t fac_empty[kScaleRing];
  uint64_t drain;
  uint32_t tmem_base;
};
constexpr size_t kSmemBytes = sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "fits one SM's shared memory");

__device__ __forceinline__ int32_t units_of(const Tile& t) {
  return (min(t.rows, kTok) + kUnit - 1) / kUnit;
}

// Positions in the rings, common to a tile's steps.
struct Rings {
  uint32_t b = 0;              // accumulator
  uint32_t st = 0, use = 0;    // stage, its use
  uint32_t r = 0, sc_use = 0;  // entry of the factor ring, its use
  bool hold = false;           // test hook: withhold the next release
};

// A tile of which this warp has kU * 16 rows from row j0 on (kU = 0: none, it
// only keeps step); false if a wait expired.
template <int kU>
__device__ __forceinline__ bool tile_body(const Params& p, Smem& s, const Tile& t, Rings& x,
                                          uint32_t tmem0, int32_t j0, int q, int lane,
                                          uint64_t wait_ns) {
  constexpr int kN = kU > 0 ? kU : 1;
  float acc[kN][kUnit];
#pragma unroll
  for (int a = 0; a < kN * kUnit; ++a) acc[a / kUnit][a % kUnit] = 0.0f;
  const uint32_t done = smem_addr(s.done), fac_full = smem_addr(s.fac_full);
  const uint32_t factors = smem_addr(s.factor), acc_empty = smem_addr(s.acc_empty);
#pragma unroll 1
  for (int32_t kb = 0; kb < p.kbs; ++kb) {
    const uint32_t e = kb % kScaleKb;
    if (e == 0 && !mbar_wait_warp(fac_full + x.r * 8, x.sc_use & 1, wait_ns, p.err)) return false;
    if (!mbar_wait_warp(done + x.st * 8, x.use & 1, wait_ns, p.err)) return false;
    tc_fence_after();
    uint32_t h[kN][kUnit];
#pragma unroll
    for (int u = 0; u < kU; ++u) tmem_ld_32x32b_x16(tmem0 + x.b * kTok + j0 + u * kUnit, h[u]);
#pragma unroll
    for (int u = 0; u < kU; ++u) tmem_ld_wait16(h[u]);
    tc_fence_before();
    __syncwarp();
    if (lane == 0 && !x.hold) mbar_arrive_addr(acc_empty + x.b * 8);
    x.hold = false;
    const uint32_t fac = factors + ((x.r * kScaleKb + e) * kTok + j0) * 4;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      uint4 f[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) f[v] = lds128_ordered(fac + (u * kUnit + 4 * v) * 4);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float w[4] = {__uint_as_float(f[v].x), __uint_as_float(f[v].y),
                            __uint_as_float(f[v].z), __uint_as_float(f[v].w)};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[u][4 * v + j] = __fmaf_rn(__uint_as_float(h[u][4 * v + j]), w[j], acc[u][4 * v + j]);
      }
    }
    if (++x.b == kBufs) x.b = 0;
    if (++x.st == kStages) {
      x.st = 0;
      ++x.use;
    }
    if (e == kScaleKb - 1 || kb == p.kbs - 1) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.fac_empty[x.r]);
      if (++x.r == kScaleRing) {
        x.r = 0;
        ++x.sc_use;
      }
    }
  }
  // Two rows at a time: neighbouring lanes swap one value each, so that even
  // lanes hold two columns of the first row and odd lanes of the second;
  // a store covers 64 bytes of both.
  const int32_t c = t.c0 + 32 * q + (lane & ~1);
  const int32_t odd = lane & 1;
  uint16_t* dst = p.out + static_cast<int64_t>(t.m0 + j0 + odd) * p.outer + c;
#pragma unroll
  for (int u = 0; u < kU; ++u)
#pragma unroll
    for (int j = 0; j < kUnit; j += 2) {
      const float give = odd ? acc[u][j] : acc[u][j + 1];
      const float got = __shfl_xor_sync(0xffffffffu, give, 1);
      const uint32_t w = odd ? bf16x2_of(got, acc[u][j + 1]) : bf16x2_of(acc[u][j], got);
      if (j0 + u * kUnit + j + odd < t.rows && c < p.outer)
        *reinterpret_cast<uint32_t*>(dst + static_cast<int64_t>(u * kUnit + j) * p.outer) = w;
    }
  return true;
}

template <bool kT>
__global__ void __launch_bounds__(kThreads, 1)
    few_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap wmap,
               const Params p) {
  extern __shared__ uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>(smem_raw + (-smem_addr(smem_raw) & 1023u));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  const uint64_t wait_ns = 4 * p.timeout_ns;

  if (warp == kEpiWarps && lane == 0) {
    prefetch_tensormap(&amap);
    prefetch_tensormap(&wmap);
  } else if (warp == kEpiWarps + 2 && lane == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.done[i], 1);
    }
    for (int b = 0; b < kBufs; ++b) mbar_init(&s.acc_empty[b], kEpiWarps);
    for (int i = 0; i < kScaleRing; ++i) {
      mbar_init(&s.fac_full[i], 1);
      mbar_init(&s.fac_empty[i], kEpiWarps);
    }
    mbar_init(&s.drain, 1);
    fence_mbar_init();
  }
  grid_wait();
  if (warp == kEpiWarps) {
    build_tiles(p, kTok, s.tiles, lane);
  } else if (warp == kEpiWarps + 1) {
    tmem_alloc(&s.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  const int32_t tiles = s.tiles.first[p.E] * p.tiles_c;  // below 2^31: the host checks

  if (warp == kEpiWarps) {
    // ------------------------------------------------------------ loads --
    const uint64_t pol_w = policy_evict_first(), pol_a = policy_evict_last();
    const uint32_t done = smem_addr(s.done);
    uint32_t st = 0, use = 0;
    bool ok = true;
    for (int32_t i = blockIdx.x; ok && i < tiles; i += gridDim.x) {
      const Tile t = tile_of(p, s.tiles, i, kTok, kCols, lane);
      const int32_t units = units_of(t);
      const uint32_t bytes = kWBytes + units * (kUnit * kBlock);
      for (int32_t k = 0; k < p.inner; k += kBlock) {
        ok = mbar_wait_warp(done + st * 8, (use & 1) ^ 1u, wait_ns, p.err);
        if (!ok) break;
        if (elect_one()) {
          uint8_t* base = s.stage[st];
          mbar_arrive_expect_tx(&s.full[st], bytes);
          tma_load_3d(base, &wmap, kT ? t.c0 : k, kT ? k : t.c0, t.g, &s.full[st], pol_w);
          for (int u = 0; u < units; ++u)
            tma_load_2d(base + kWBytes + u * (kUnit * kBlock), &amap, k, t.m0 + u * kUnit,
                        &s.full[st], pol_a);
        }
        __syncwarp();
        if (++st == kStages) {
          st = 0;
          ++use;
        }
      }
    }
    // the block must not exit while a load is still writing its memory, also
    // after a wait that ran out; the MMAs that read it are waited for below
    for (uint32_t u = 0; u < kStages; ++u) {
      const uint32_t uses = use + (u < st ? 1 : 0);
      if (uses > 0) mbar_wait_warp(smem_addr(&s.full[u]), (uses - 1) & 1, wait_ns, p.err);
    }
  } else if (warp == kEpiWarps + 1) {
    // ------------------------------------------------------------- MMAs --
    const uint32_t acc_empty = smem_addr(s.acc_empty), full = smem_addr(s.full);
    const uint32_t stage0 = smem_addr(s.stage);
    constexpr uint32_t wstep = kT ? (kSubK * kBlock) >> 4 : kSubK >> 4;
    uint32_t st = 0, st_use = 0, b = 0, use = 0;
    bool ok = true, issued = false;
    for (int32_t i = blockIdx.x; ok && i < tiles; i += gridDim.x) {
      const Tile t = tile_of(p, s.tiles, i, kTok, kCols, lane);
      const uint32_t n = __shfl_sync(0xffffffffu, units_of(t) * kUnit, 0);
      // D fp32, e4m3 x e4m3, M = 128, A MN-major if transposed, N = n
      const uint32_t idesc = (1u << 4) | (kT ? 1u << 15 : 0u) | ((n >> 3) << 17) | (8u << 24);
      for (int32_t left = p.inner; left > 0; left -= kBlock) {
        ok = mbar_wait_warp(acc_empty + b * 8, (use & 1) ^ 1u, wait_ns, p.err) &&
             mbar_wait_warp(full + st * 8, st_use & 1, wait_ns, p.err);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t d = tmem + b * kTok, w0 = stage0 + st * kStageBytes;
          uint64_t wd = operand_desc_sw128(w0);
          uint64_t ad = operand_desc_sw128(w0 + kWBytes);
          tc_mma_e4m3<false>(d, wd, ad, idesc);
#pragma unroll
          for (int j = 1; j < kBlock / kSubK; ++j) {
            wd += wstep;
            ad += kSubK >> 4;
            if (j * kSubK < left) tc_mma_e4m3<true>(d, wd, ad, idesc);
          }
          tc_commit(&s.done[st]);
        }
        __syncwarp();
        issued = true;
        if (++b == kBufs) {
          b = 0;
          ++use;
        }
        if (++st == kStages) {
          st = 0;
          ++st_use;
        }
      }
    }
    // every MMA is complete before the TMEM is freed
    if (issued) {
      if (elect_one()) tc_commit(&s.drain);
      __syncwarp();
      mbar_wait_warp(smem_addr(&s.drain), 0, wait_ns, p.err);
    }
  } else if (warp == kEpiWarps + 2) {
    // ---------------------------------------------------------- factors --
    // the scales of an entry are loaded while the one before is worked on
    float v[kTok / 32][kScaleKb] = {}, w[kScaleKb];
    int32_t i = blockIdx.x, kb = 0, rows = 0;
    Tile t = {};
    auto load = [&]() {  // the entry (tile i, 128-blocks kb ..)
      if (kb == 0) t = tile_of(p, s.tiles, i, kTok, kCols, lane);
      rows = min(t.rows, kTok);
      const float* sb = p.sb + t.g * p.sb_expert +
                        static_cast<int64_t>(min(t.c0 / kBlock, p.sb_last)) * p.sb_c;
#pragma unroll
      for (int u = 0; u < kScaleKb; ++u)
        w[u] = __ldg(sb + static_cast<int64_t>(min(kb + u, p.kbs - 1)) * p.sb_k);
#pragma unroll
      for (int j = 0; j < kTok / 32; ++j) {
        if (lane + 32 * j >= rows) break;
        const float* sa = p.sa + static_cast<int64_t>(t.m0 + lane + 32 * j) * p.kbs;
        if (p.sa_vec) {
          const float4 x = __ldg(reinterpret_cast<const float4*>(sa + kb));
          v[j][0] = x.x;
          v[j][1] = x.y;
          v[j][2] = x.z;
          v[j][3] = x.w;
        } else {
#pragma unroll
          for (int u = 0; u < kScaleKb; ++u) v[j][u] = __ldg(sa + min(kb + u, p.kbs - 1));
        }
      }
    };
    const uint32_t empty = smem_addr(s.fac_empty);
    uint32_t r = 0, use = 0;
    bool ok = true;
    if (i < tiles) load();
    while (i < tiles) {
      float f[kTok / 32][kScaleKb];
#pragma unroll
      for (int u = 0; u < kScaleKb; ++u) {
        const float rw = rcp_approx(w[u]);
#pragma unroll
        for (int j = 0; j < kTok / 32; ++j) f[j][u] = __fmul_rn(rcp_approx(v[j][u]), rw);
      }
      const int32_t have = rows;
      kb += kScaleKb;
      if (kb >= p.kbs) {
        kb = 0;
        i += gridDim.x;
      }
      if (i < tiles) load();
      ok = mbar_wait_warp(empty + r * 8, (use & 1) ^ 1u, wait_ns, p.err);
      if (!ok) break;
#pragma unroll
      for (int j = 0; j < kTok / 32; ++j)
        if (lane + 32 * j < have)
#pragma unroll
          for (int u = 0; u < kScaleKb; ++u) s.factor[r][u][lane + 32 * j] = f[j][u];
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.fac_full[r]);
      if (++r == kScaleRing) {
        r = 0;
        ++use;
      }
    }
  } else {
    // --------------------------------------------------------- epilogue --
    const int q = warp & 3;
    const uint32_t tmem0 = tmem + (static_cast<uint32_t>(32 * q) << 16);
    const int32_t j0 = (warp >> 2) * kWarpTok;
    Rings x;
    x.hold = p.skip_arrival && blockIdx.x == 0;
    bool ok = true;
    for (int32_t i = blockIdx.x; ok && i < tiles; i += gridDim.x) {
      const Tile t = tile_of(p, s.tiles, i, kTok, kCols, lane);
      switch (min(units_of(t) - j0 / kUnit, kWarpTok / kUnit)) {
        case 4: ok = tile_body<4>(p, s, t, x, tmem0, j0, q, lane, wait_ns); break;
        case 3: ok = tile_body<3>(p, s, t, x, tmem0, j0, q, lane, wait_ns); break;
        case 2: ok = tile_body<2>(p, s, t, x, tmem0, j0, q, lane, wait_ns); break;
        case 1: ok = tile_body<1>(p, s, t, x, tmem0, j0, q, lane, wait_ns); break;
        default: ok = tile_body<0>(p, s, t, x, tmem0, j0, q, lane, wait_ns); break;
      }
    }
    tc_fence_before();
  }

  __syncthreads();
  if (warp == kEpiWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

gq_status setup_few(DeviceInfo& info) {
  (void)info;
  for (const void* f : {reinterpret_cast<const void*>(few_kernel<false>),
                        reinterpret_cast<const void*>(few_kernel<true>)}) {
    const gq_status st = check_cuda(
        cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmemBytes)),
        "grouped_mm: shared memory size");
    if (st != GQ_OK) return st;
  }
  return GQ_OK;
}

gq_status launch_few(const DeviceInfo& info, Params p, const void* qa, const void* qb,
                     int32_t N, int32_t K, cudaStream_t stream) {
  CUtensorMap amap, wmap;
  gq_status st = encode_tiled_2d(&amap, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<void*>(qa),
                                 static_cast<uint64_t>(p.inner), static_cast<uint64_t>(p.M),
                                 static_cast<uint64_t>(p.inner), kBlock, kUnit,
                                 CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != GQ_OK) return st;
  st = encode_tiled_3d(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<void*>(qb),
                       static_cast<uint64_t>(K), static_cast<uint64_t>(N),
                       static_cast<uint64_t>(p.E), static_cast<uint64_t>(K),
                       static_cast<uint64_t>(N) * K, kBlock, kBlock, CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != GQ_OK) return st;
  p.tiles_c = (p.outer + kCols - 1) / kCols;
  const int64_t most =
      (static_cast<int64_t>(p.M) / kTok + (p.E < p.M ? p.E : p.M)) * p.tiles_c;  // any offsets
  if (most > INT32_MAX)
    return fail(GQ_ERR_UNSUPPORTED, "grouped_mm: %lld tiles", static_cast<long long>(most));
  const unsigned grid = static_cast<unsigned>(most < info.sm_count ? most : info.sm_count);
  const auto kernel = p.transposed ? few_kernel<true> : few_kernel<false>;
  return launch_chained("grouped_mm: launch", kernel, dim3(grid), kThreads, kSmemBytes, stream, 1,
                        amap, wmap, p);
}

}  // namespace gmm
}  // namespace gq
