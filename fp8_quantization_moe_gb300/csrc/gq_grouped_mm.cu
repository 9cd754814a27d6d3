// gq_grouped_mm.cu -- the grouped product of block-quantized rows with
// block-quantized stacked weights, one expert per token group, on the
// sm_103a tensor cores (tcgen05 in block pairs, TMEM accumulators, TMA):
//   forward     out[m][n] = sum_k A[m][k] * W[e][n][k]
//   transposed  out[m][k] = sum_n A[m][n] * W[e][n][k]
// with A = qa / sa (one scale per row and 128 contraction columns) and
// W = qb / sb (one scale per 128x128 block).  Within a 128-block kb of the
// contraction both scales are constant for a row m and 128 output columns c,
//   out[m][c] = sum_kb ( 1/sa[m][kb] * 1/sb[e][c/128, kb] ) * P_kb[m][c],
// P_kb the plain sum of the block's e4m3 products.  The tensor cores form
// P_kb in TMEM (fp32); the epilogue warps read it, multiply by the factor
// and add it to fp32 accumulators in registers, rounded to bf16 once.
//
// Two blocks of a cluster share a tile of 256 rows x 256 output columns
// (cta_group::2): each loads 128 of the rows and 128 of the weights' rows or
// columns, 128 contraction columns at a time, and the pair's MMAs read both
// halves: per block and 128-block 32 KB enter the shared memory and 32 KB
// leave it, 512 cycles at 128 bytes a cycle and as many of MMA work.  (One
// block alone would need 48 KB for the same work.)
//
// The rows are the MMA's M operand, so that a TMEM lane is a row and its
// factor one register: with the weights as M a lane would need every row's
// factor, and those loads alone -- shared memory returns 128 bytes a cycle --
// would cost as much as the MMAs.  A group's last tile pays for 256 rows.
//
// Warp roles, per block:
//   0-7   epilogue: lane quarter w % 4 (32 rows), column half w / 4;
//   8     TMA loads (one lane);
//   9     TMEM allocation; in the pair's first block the MMAs (one lane);
//   10    copies the scales of the next 128-blocks into a ring in shared memory
//         (loads by the warps that use them would be microseconds late under
//         the TMA traffic: 490 -> 550 us for the case below);
//   11    idle: it completes the warpgroup whose registers 0-7 take over.
// Every mbarrier wait is bounded; on expiry the error word is set, the warp
// leaves its loop and the others time out in turn.
#include <cuda_bf16.h>

#include "gq_grouped_mm.cuh"
#include "gq_tcgen05.cuh"

namespace gq {
namespace gmm {

constexpr int kRows = 128;        // rows per block of a pair
constexpr int kCols = 256;        // output columns of a tile
constexpr int kBoxRows = 32;      // rows per TMA box where a block has few
constexpr int kStages = 6;
constexpr int kABytes = kRows * kBlock;        // 16 KB
constexpr int kWBytes = kCols / 2 * kBlock;    // 16 KB
constexpr int kStageBytes = kABytes + kWBytes;
constexpr int kBufs = 2;          // accumulators in TMEM
constexpr uint32_t kTmemCols = kBufs * kCols;
constexpr int kEpiWarps = 8;      // two per TMEM lane quarter
constexpr int kThreads = (kEpiWarps + 4) * 32;
constexpr int kChunk = 32;        // columns per step of the epilogue
constexpr int kChunks = kCols / 2 / kChunk;
constexpr int kScaleKb = 4;       // 128-blocks per entry of the scale ring
constexpr int kScaleRing = 4;
#ifndef FEW
#define FEW 32
#endif
constexpr int kFewRows = FEW;
static_assert(kTmemCols == 512 && kChunks == 4, "two accumulators fill the TMEM");

struct Smem {
  uint8_t stage[kStages][kStageBytes];  // 1024-byte aligned (swizzle atoms)
  alignas(16) uint8_t rows[kEpiWarps][32 * kChunk * 2];
  alignas(16) float sa[kScaleRing][kRows][kScaleKb];  // of the block's rows
  alignas(16) float sb[kScaleRing][2][kScaleKb];      // of the tile's two column halves
  TileTable tiles;
  uint64_t full[kStages];         // both blocks' loads (the pair's first block)
  uint64_t done[kStages];         // the stage's MMAs are complete (commit, both blocks):
                                  // the stage is free, its accumulator full
  uint64_t acc_empty[kBufs];      // accumulator read (16 warps; the first block)
  uint64_t sc_full[kScaleRing];   // scales copied (warp 10)
  uint64_t sc_empty[kScaleRing];  // scales read (8 warps)
  uint64_t drain;
  uint32_t tmem_base;
};
constexpr size_t kSmemBytes = sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "fits one SM's shared memory");

// Rows of the tile that block `rank` of the pair holds.
__device__ __forceinline__ int32_t rows_of(const Tile& t, int32_t rank) {
  return min(max(t.rows - rank * kRows, 0), kRows);
}
// TMA boxes of kBoxRows rows for them (4: one box of kRows).
__device__ __forceinline__ int32_t boxes_of(int32_t rows) {
  return (rows + kBoxRows - 1) / kBoxRows;
}

// The MMA's N: the tile's columns in steps of 32, as the pair form takes them.
// A block's half is then a multiple of 16 columns: in the transposed product,
// where columns are the innermost coordinate, a TMA box may start there.
__device__ __forceinline__ int32_t mma_cols(const Params& p, const Tile& t) {
  return min((p.outer - t.c0 + 31) & ~31, kCols);
}

// acc += h * f, h the bits of fp32 values.  (Scalar multiply-adds: the packed
// form reads twice the registers and, next to TMEM loads, measured 54 cycles
// for 32 columns against 39.)
__device__ __forceinline__ void scale_add(float (&acc)[kChunk], const uint32_t (&h)[kChunk],
                                          float f) {
#pragma unroll
  for (int e = 0; e < kChunk; ++e) acc[e] = __fmaf_rn(__uint_as_float(h[e]), f, acc[e]);
}

// D fp32, e4m3 x e4m3, M = 256; A K-major, B K-major unless transposed (bit 16).
constexpr uint32_t kIdescBase = (1u << 4) | (16u << 24);

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap amap,
                   const __grid_constant__ CUtensorMap amap32,
                   const __grid_constant__ CUtensorMap wmap, const Params p) {
  // aligned by an offset, so that the compiler still knows the address space
  extern __shared__ uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>(smem_raw + (-smem_addr(smem_raw) & 1023u));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const uint64_t wait_ns = 4 * p.timeout_ns;

  if (warp == kEpiWarps) {
    build_tiles(p, 2 * kRows, s.tiles, lane);
    if (lane == 0) {
      prefetch_tensormap(&amap);
      prefetch_tensormap(&amap32);
      prefetch_tensormap(&wmap);
    }
  } else if (warp == kEpiWarps + 1) {
    tmem_alloc_pair(&s.tmem_base, kTmemCols);
    tmem_relinquish_pair();
  } else if (warp == kEpiWarps + 2 && lane == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.done[i], 1);
    }
    for (int b = 0; b < kBufs; ++b) mbar_init(&s.acc_empty[b], 2 * kEpiWarps);
    for (int i = 0; i < kScaleRing; ++i) {
      mbar_init(&s.sc_full[i], 32);
      mbar_init(&s.sc_empty[i], kEpiWarps);
    }
    mbar_init(&s.drain, 1);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive();  // the peer's barriers are ready as well
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  const int32_t tiles = s.tiles.first[p.E] * p.tiles_c;  // below 2^31: the host checks
  const int32_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (warp >= kEpiWarps) {
    setmaxnreg_dec<40>();
    if (warp == kEpiWarps) {
      // ---------------------------------------------------------- loads --
      const uint64_t pol = policy_evict_normal();
      const uint32_t done = smem_addr(s.done), full = map_cluster(smem_addr(s.full), 0);
      uint32_t st = 0, use = 0;  // stage, its use
      bool ok = true;
      for (int32_t i = pair; ok && i < tiles; i += pairs) {
        const Tile t = tile_of(p, s.tiles, i, 2 * kRows, kCols);
        const int32_t boxes = boxes_of(rows_of(t, rank));
        const uint32_t bytes = 2u * kWBytes + static_cast<uint32_t>(
            boxes_of(rows_of(t, 0)) + boxes_of(rows_of(t, 1))) * (kBoxRows * kBlock);
        const int32_t m = t.m0 + static_cast<int32_t>(rank) * kRows;
        const int32_t c = t.c0 + static_cast<int32_t>(rank) * (mma_cols(p, t) / 2);
        for (int32_t k = 0; k < p.inner; k += kBlock) {
          ok = mbar_wait_warp(done + st * 8, (use & 1) ^ 1u, wait_ns, p.err);
          if (!ok) break;
          if (elect_one()) {
            uint8_t* base = s.stage[st];
            if (rank == 0)  // both blocks' bytes complete on the first block's barrier
              mbar_arrive_expect_tx(&s.full[st], bytes);
            const uint32_t bar = full + st * 8;
            tma_load_3d_pair(base + kABytes, &wmap, p.transposed ? c : k, p.transposed ? k : c, t.g,
                             bar, pol);
            if (boxes == kRows / kBoxRows)
              tma_load_2d_pair(base, &amap, k, m, bar, pol);
            else
              for (int b = 0; b < boxes; ++b)
                tma_load_2d_pair(base + b * kBoxRows * kBlock, &amap32, k, m + b * kBoxRows, bar,
                                 pol);
          }
          __syncwarp();
          if (++st == kStages) {
            st = 0;
            ++use;
          }
        }
      }
      // every load has landed and been read before the block may exit
      for (uint32_t u = 0; ok && u < kStages; ++u) {
        const uint32_t uses = use + (u < st ? 1 : 0);
        if (uses > 0) ok = mbar_wait_warp(done + u * 8, (uses - 1) & 1, wait_ns, p.err);
      }
    } else if (warp == kEpiWarps + 1) {
      // ----------------------------------------------------------- MMAs --
      if (rank == 0) {
        const uint32_t acc_empty = smem_addr(s.acc_empty), full = smem_addr(s.full);
        const uint32_t stage0 = smem_addr(s.stage);
        const uint32_t wstep = p.transposed ? (kSubK * kBlock) >> 4 : kSubK >> 4;
        uint32_t st = 0, st_use = 0, b = 0, use = 0;  // stage and accumulator, their uses
        bool ok = true, issued = false;
        for (int32_t i = pair; ok && i < tiles; i += pairs) {
          const Tile t = tile_of(p, s.tiles, i, 2 * kRows, kCols);
          const uint32_t n = __shfl_sync(0xffffffffu, mma_cols(p, t), 0);
          const uint32_t idesc = kIdescBase | ((n >> 3) << 17) | (p.transposed ? 1u << 16 : 0u);
          for (int32_t left = p.inner; left > 0; left -= kBlock) {
            const bool loaded = mbar_test_addr(full + st * 8, st_use & 1);
            ok = mbar_wait_warp(acc_empty + b * 8, (use & 1) ^ 1u, wait_ns, p.err) &&
                 (__all_sync(0xffffffffu, loaded) ||
                  mbar_wait_warp(full + st * 8, st_use & 1, wait_ns, p.err));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              const uint32_t d = tmem + b * kCols;
              // rows: K-major; weights: K-major rows of 128 bytes, or
              // MN-major (32 contraction rows = 4 KB)
              const uint32_t a0 = stage0 + st * kStageBytes;
              uint64_t ad = operand_desc_sw128(a0);
              uint64_t wd = operand_desc_sw128(a0 + kABytes);
              tc_mma_e4m3_pair<false>(d, ad, wd, idesc);
#pragma unroll
              for (int j = 1; j < kBlock / kSubK; ++j) {
                ad += kSubK >> 4;
                wd += wstep;
                if (j * kSubK < left) tc_mma_e4m3_pair<true>(d, ad, wd, idesc);
              }
              tc_commit_pair(&s.done[st], 3);
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
          if (elect_one()) tc_commit_pair(&s.drain, 1);
          __syncwarp();
          mbar_wait_warp(smem_addr(&s.drain), 0, wait_ns, p.err);
        }
      }
      __syncwarp();
    } else if (warp == kEpiWarps + 2) {
      // --------------------------------------------------------- scales --
      const uint32_t empty = smem_addr(s.sc_empty);
      uint32_t r = 0, use = 0;  // entry, its use
      bool ok = true;
      for (int32_t i = pair; ok && i < tiles; i += pairs) {
        const Tile t = tile_of(p, s.tiles, i, 2 * kRows, kCols);
        // only rows that exist: clamped to one row, the copies of all blocks
        // would queue up at a single L2 line (20 us for a product of 8 rows)
        const int32_t rows = rows_of(t, rank);
        const float* src = p.sa +
            static_cast<int64_t>(t.m0 + static_cast<int32_t>(rank) * kRows + lane) * p.kbs;
        // lane = 4 * half + 128-block
        const float* sb = p.sb + t.g * p.sb_expert +
            static_cast<int64_t>(min(t.c0 / kBlock + (lane >> 2), p.sb_last)) * p.sb_c;
        for (int32_t kb = 0; kb < p.kbs; kb += kScaleKb) {
          ok = mbar_wait_warp(empty + r * 8, (use & 1) ^ 1u, wait_ns, p.err);
          if (!ok) break;
          for (int j = 0; lane + j < rows; j += 32) {
            const uint32_t dst = smem_addr(s.sa[r][lane + j]);
            const float* from = src + static_cast<int64_t>(j) * p.kbs;
            if (p.sa_vec)
              cp_async_16(dst, from + kb, 16);
            else
              for (int u = 0; u < kScaleKb; ++u)
                cp_async_4(dst + 4 * u, from + min(kb + u, p.kbs - 1));
          }
          __syncwarp();
          if (lane < 2 * kScaleKb)
            cp_async_4(smem_addr(s.sb[r][lane >> 2]) + 4 * (lane & 3),
                       sb + static_cast<int64_t>(min(kb + (lane & 3), p.kbs - 1)) * p.sb_k);
          cp_async_mbar_arrive(&s.sc_full[r]);
          mbar_arrive(&s.sc_full[r]);
          if (++r == kScaleRing) {
            r = 0;
            ++use;
          }
        }
      }
      // the copies have landed and been read before the block may exit
      for (uint32_t u = 0; ok && u < kScaleRing; ++u) {
        const uint32_t uses = use + (u < r ? 1 : 0);
        if (uses > 0) ok = mbar_wait_warp(empty + u * 8, (uses - 1) & 1, wait_ns, p.err);
      }
    }
  } else {
    // --------------------------------------------------------- epilogue --
    // Lane l of warp (q, hc) owns row 32 q + l of its block's rows and the
    // tile's columns [128 hc, 128 hc + 128), one scale block of the weights.
    setmaxnreg_inc<232>();
    const int q = warp & 3, hc = warp >> 2;
    const uint32_t stage_rows = smem_addr(s.rows[warp]);
    const uint32_t my_row = stage_rows + static_cast<uint32_t>(lane * kChunk * 2);
    const uint32_t my_swz = static_cast<uint32_t>((lane >> 1) & 3);
    const uint32_t done = smem_addr(s.done);
    const uint32_t acc_empty = map_cluster(smem_addr(s.acc_empty), 0);
    const uint32_t tmem0 = tmem + (static_cast<uint32_t>(32 * q) << 16) + hc * (kCols / 2);
    uint32_t b = 0;             // accumulator
    uint32_t st = 0, use = 0;   // the stage whose MMAs filled it, its use
    const uint32_t sc_full = smem_addr(s.sc_full);
    const uint32_t sc_a = smem_addr(s.sa[0][32 * q + lane]), sc_w = smem_addr(s.sb[0][hc]);
    uint32_t r = 0, sc_use = 0;  // entry of the scale ring, its use
    bool ready = false;         // its MMAs are known to be complete
    bool first = p.skip_arrival && blockIdx.x == 0;  // withhold the next release
    bool ok = true;
    for (int32_t i = pair; ok && i < tiles; i += pairs) {
      const Tile t = tile_of(p, s.tiles, i, 2 * kRows, kCols);
      const int32_t rows = rows_of(t, rank) - 32 * q;  // of this warp, if positive
      const int32_t c = t.c0 + hc * (kCols / 2);
      const bool mine = rows > 0 && c < p.outer;
      const int32_t row = t.m0 + static_cast<int32_t>(rank) * kRows + 32 * q + lane;
      float acc[kChunks][kChunk];
#pragma unroll
      for (int a = 0; a < kChunks * kChunk; ++a) acc[a / kChunk][a % kChunk] = 0.0f;
      // one 128-block per turn, not unrolled: the code of a turn is fetched
      // once (unrolled four times, a launch spent 20 us on fetching it)
#pragma unroll 1
      for (int32_t kb = 0; kb < p.kbs; ++kb) {
        const uint32_t e = kb % kScaleKb;
        if (e == 0) {
          ok = mbar_wait_warp(sc_full + r * 8, sc_use & 1, wait_ns, p.err);
          if (!ok) break;
        }
        const float f =
            __fmul_rn(rcp_approx(lds32_ordered(sc_a + r * (kRows * kScaleKb * 4) + e * 4)),
                      rcp_approx(lds32_ordered(sc_w + r * (2 * kScaleKb * 4) + e * 4)));
        if (e == kScaleKb - 1 || kb == p.kbs - 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.sc_empty[r]);
          if (++r == kScaleRing) {
            r = 0;
            ++sc_use;
          }
        }
        if (!__all_sync(0xffffffffu, ready)) {
          ok = mbar_wait_warp(done + st * 8, use & 1, wait_ns, p.err);
          if (!ok) break;
        }
        tc_fence_after();
        const uint32_t tacc = tmem0 + b * kCols;
        uint32_t h0[kChunk], h1[kChunk];
        if (mine) {
          tmem_ld_32x32b_x32(tacc, h0);
          tmem_ld_32x32b_x32(tacc + kChunk, h1);
          tmem_ld_wait32(h0);
          tmem_ld_wait32(h1);
          scale_add(acc[0], h0, f);
          tmem_ld_32x32b_x32(tacc + 2 * kChunk, h0);
          scale_add(acc[1], h1, f);
          tmem_ld_32x32b_x32(tacc + 3 * kChunk, h1);
          tmem_ld_wait32(h0);
          tmem_ld_wait32(h1);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && !first) mbar_arrive_cluster(acc_empty + b * 8);
        first = false;
        b ^= 1;
        if (++st == kStages) {
          st = 0;
          ++use;
        }
        // the answer arrives behind the arithmetic
        ready = mbar_test_addr(done + st * 8, use & 1);
        if (mine) {
          scale_add(acc[2], h0, f);
          scale_add(acc[3], h1, f);
        }
      }
      if (!ok) break;
      if (!mine) continue;
      // 32 columns at a time: each lane writes its row's 64-byte run into the
      // warp's staging rows (16-byte parts XOR-swizzled by (row / 2) % 4: no
      // bank conflicts on either side), then eight rows per store
      const int part = lane & 3;
      uint16_t* orow = p.out + static_cast<int64_t>(row - lane) * p.outer + c + part * 8;
#pragma unroll
      for (int ch = 0; ch < kChunks; ++ch) {
        if (c + ch * kChunk >= p.outer) break;
#pragma unroll
        for (int w = 0; w < 4; ++w)
          sts128(my_row + ((static_cast<uint32_t>(w) ^ my_swz) << 4),
                 make_uint4(bf16x2_of(acc[ch][8 * w], acc[ch][8 * w + 1]),
                            bf16x2_of(acc[ch][8 * w + 2], acc[ch][8 * w + 3]),
                            bf16x2_of(acc[ch][8 * w + 4], acc[ch][8 * w + 5]),
                            bf16x2_of(acc[ch][8 * w + 6], acc[ch][8 * w + 7])));
        __syncwarp();
        const bool c_ok = c + ch * kChunk + part * 8 < p.outer;  // outer % 16 == 0
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int m = 8 * k + (lane >> 2);
          const uint4 v = lds128_ordered(stage_rows + m * (kChunk * 2) + ((part ^ ((m >> 1) & 3)) << 4));
          if (m < rows && c_ok)
            *reinterpret_cast<uint4*>(orow + static_cast<int64_t>(m) * p.outer + ch * kChunk) = v;
        }
        __syncwarp();
      }
    }
    tc_fence_before();
  }

  __syncthreads();
  cluster_arrive();  // neither block leaves while the other may still signal it
  cluster_wait();
  if (warp == kEpiWarps + 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

gq_status setup(DeviceInfo& info) {
  gq_status st = check_cuda(
      cudaFuncSetAttribute(product_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kSmemBytes)),
      "grouped_mm: shared memory size");
  if (st != GQ_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(info.sm_count / 2 * 2));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int pairs = 0;
  st = check_cuda(cudaOccupancyMaxActiveClusters(&pairs, product_kernel, &cfg),
                  "grouped_mm: resident block pairs");
  if (st != GQ_OK) return st;
  info.mm_pairs = pairs > 0 ? pairs : 1;
  return setup_few(info);
}

gq_status launch(const DeviceInfo& info, const DebugKnobs& dbg, const void* qa, const float* sa,
                 int64_t M, const void* qb, const float* sb, int32_t N, int32_t K, bool transposed,
                 const int32_t* offs, int32_t E, void* out, cudaStream_t stream) {
  const int32_t nb_n = (N + kBlock - 1) / kBlock, nb_k = (K + kBlock - 1) / kBlock;
  Params p;
  p.inner = transposed ? N : K;
  p.outer = transposed ? K : N;
  p.sa = sa;
  p.sb = sb;
  p.offs = offs;
  p.out = static_cast<uint16_t*>(out);
  p.err = info.err_word;
  p.M = static_cast<int32_t>(M);
  p.E = E;
  p.kbs = (p.inner + kBlock - 1) / kBlock;
  p.tiles_c = (p.outer + kCols - 1) / kCols;
  p.sb_expert = static_cast<int64_t>(nb_n) * nb_k;
  p.sb_c = transposed ? 1 : nb_k;
  p.sb_k = transposed ? nb_k : 1;
  p.sb_last = (transposed ? nb_k : nb_n) - 1;
  p.sa_vec = p.kbs % kScaleKb == 0 && (reinterpret_cast<uintptr_t>(sa) & 15) == 0;
  p.transposed = transposed;
  p.timeout_ns = dbg.timeout_ns;
  p.skip_arrival = dbg.skip_arrival;
  if (M <= static_cast<int64_t>(kFewRows) * E) return launch_few(info, p, qa, qb, N, K, stream);

  const int64_t most = (M / (2 * kRows) + (E < M ? E : M)) * p.tiles_c;  // tiles of any offsets
  if (most > INT32_MAX)
    return fail(GQ_ERR_UNSUPPORTED, "grouped_mm: %lld tiles", static_cast<long long>(most));
  CUtensorMap amap, amap32, wmap;
  gq_status st = GQ_OK;
  for (CUtensorMap* m : {&amap, &amap32}) {
    st = encode_tiled_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<void*>(qa),
                         static_cast<uint64_t>(p.inner), static_cast<uint64_t>(M),
                         static_cast<uint64_t>(p.inner), kBlock, m == &amap ? kRows : kBoxRows,
                         CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != GQ_OK) return st;
  }
  // three dimensions: rows and columns past an expert's own read zeros, never
  // the next expert's (a NaN there would survive the product with zero)
  st = encode_tiled_3d(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<void*>(qb),
                       static_cast<uint64_t>(K), static_cast<uint64_t>(N), static_cast<uint64_t>(E),
                       static_cast<uint64_t>(K), static_cast<uint64_t>(N) * K, kBlock, kBlock,
                       CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != GQ_OK) return st;
  const int64_t pairs = most < info.mm_pairs ? most : info.mm_pairs;
  product_kernel<<<static_cast<unsigned>(2 * pairs), kThreads, kSmemBytes, stream>>>(amap, amap32,
                                                                                     wmap, p);
  return check_cuda(cudaGetLastError(), "grouped_mm: launch");
}

}  // namespace gmm
}  // namespace gq
