// gq_grouped_mm.cu -- the grouped product of block-quantized rows with
// block-quantized stacked weights, one expert per token group, on the
// sm_103a tensor cores (tcgen05, TMEM accumulators, TMA operands):
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
// A block takes tiles of 128 rows x 256 output columns, 128 contraction
// columns at a time.  The rows are the MMA's M operand, so that a TMEM lane
// is a row and its factor one register: with the weights as M a lane would
// need every row's factor, and those loads alone -- shared memory returns 128
// bytes a cycle -- would cost as much as the MMAs.
//
// What bounds it: the tensor cores work for 512 of a 128-block's 860 cycles.
// With two accumulators, all of TMEM, the MMAs wait for the epilogue: without
// its multiply-adds (half of the FMA pipe's time at the tensor cores' full
// rate) a 128-block would take 720 cycles, without the stores 780: a tile's 64
// KB leave the SM at 32 bytes a cycle, and for those 2000 cycles the MMAs run
// ahead by two 128-blocks at most.  Without multiply-adds and TMEM loads 700 are
// left, 188 above the MMAs; what of that the stores do not explain is not known.
// 16,640 rows of 16 groups, K 4096 to N 8192: 460 us, 2.43 PFLOP/s; transposed,
// 32,768 rows of 64 groups, N 2048 to K 4096: 265 us, 2.07 PFLOP/s; in a long
// run, at the power limit's clock, 515 to 540 and 295 to 311 us.  Blocks in pairs
// that share the weights' loads (cta_group::2) release accumulators across
// blocks and pad the groups to 256 rows: 505 and 316 us when this kernel took
// 485 and 284 (long runs 536 and 330 against 528 and 304); they were not
// measured with what has made it faster since.
//
// One persistent block per SM; its warps:
//   0-7   epilogue: lane quarter w % 4 (32 rows), column half w / 4;
//   8     TMA loads (one lane);
//   9     TMEM allocation and the MMAs (one lane);
//   10-11 the factors 1/sa * 1/sb, 64 rows each, four 128-blocks at a time,
//         into a ring in shared memory.
// Every mbarrier wait is bounded; on expiry the error word is set, the warp
// leaves its loop and the others time out in turn.
#include <cuda_bf16.h>

#include "gq_grouped_mm.cuh"
#include "gq_tcgen05.cuh"

namespace gq {
namespace gmm {
namespace {

constexpr int kRows = 128;        // rows of a tile
constexpr int kCols = 256;        // output columns of a tile
constexpr int kBoxRows = 32;      // rows per TMA box where a tile has few
constexpr int kStages = 4;
constexpr int kABytes = kRows * kBlock;        // 16 KB
constexpr int kWHalf = kCols / 2 * kBlock;     // 16 KB: 128 output columns
constexpr int kStageBytes = kABytes + 2 * kWHalf;
constexpr int kBufs = 2;          // accumulators in TMEM
constexpr uint32_t kTmemCols = kBufs * kCols;
constexpr int kEpiWarps = 8;      // two per TMEM lane quarter
constexpr int kThreads = (kEpiWarps + 4) * 32;
constexpr int kEpiRegs = 232;     // registers per thread after the split:
constexpr int kOtherRegs = 40;    // what the block was launched with, no more
constexpr int kChunk = 32;        // columns per step of the epilogue
constexpr int kChunks = kCols / 2 / kChunk;
constexpr int kScaleKb = 4;       // 128-blocks per entry of the factor ring
constexpr int kScaleRing = 2;
static_assert(kTmemCols == 512 && kChunks == 4, "two accumulators fill the TMEM");

struct Smem {
  uint8_t stage[kStages][kStageBytes];  // 1024-byte aligned (swizzle atoms)
  float factor[kScaleRing][kScaleKb][2][kRows];  // of the tile's two column halves
  int4 tile[kScaleRing];         // the entry's tile: first row, rows, first column
  uint32_t cols[kStages];        // output columns of the stage's tile
  TileTable tiles;
  uint64_t full[kStages];         // the stage's loads
  uint64_t done[kStages];         // its MMAs are complete: the stage is free, the accumulator full
  uint64_t acc_empty[kBufs];      // accumulator read (8 warps)
  uint64_t fac_full[kScaleRing];  // factors written (2 warps)
  uint64_t fac_empty[kScaleRing]; // factors read (8 warps)
  uint64_t drain;
  uint32_t tmem_base;
};
constexpr size_t kSmemBytes = sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "fits one SM's shared memory");

// TMA boxes of kBoxRows rows for a tile's rows (4: one box of kRows).
__device__ __forceinline__ int32_t boxes_of(const Tile& t) {
  return (min(t.rows, kRows) + kBoxRows - 1) / kBoxRows;
}

// acc += h * f, h the bits of fp32 values, two at a time.  A packed multiply-
// add occupies the FMA pipe for as long as two scalar ones (measured 2 cycles)
// but issues once: with scalar ones the warp that issues the MMAs waits for
// its turn (500 us instead of 488 for 16,640 rows).
__device__ __forceinline__ void scale_add(float (&acc)[kChunk], const uint32_t (&h)[kChunk],
                                          float f) {
#pragma unroll
  for (int e = 0; e < kChunk; e += 2) fma2(acc[e], acc[e + 1], h[e], h[e + 1], f);
}

// Exchanges b of a lane without bit kD with a of its partner with that bit.
template <int kD>
__device__ __forceinline__ void swap_with(uint32_t& a, uint32_t& b, int lane) {
  const bool up = (lane & kD) != 0;
  const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? a : b, kD);
  if (up)
    a = got;
  else
    b = got;
}

template <bool kT>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap amap,
                   const __grid_constant__ CUtensorMap amap32,
                   const __grid_constant__ CUtensorMap wmap, const Params p) {
  // aligned by an offset, so that the compiler still knows the address space
  extern __shared__ uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>(smem_raw + (-smem_addr(smem_raw) & 1023u));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  const uint64_t wait_ns = 4 * p.timeout_ns;

  if (warp == kEpiWarps && lane == 0) {
    prefetch_tensormap(&amap);
    prefetch_tensormap(&amap32);
    prefetch_tensormap(&wmap);
  } else if (warp == kEpiWarps + 2 && lane == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.done[i], 1);
    }
    for (int b = 0; b < kBufs; ++b) mbar_init(&s.acc_empty[b], kEpiWarps);
    for (int i = 0; i < kScaleRing; ++i) {
      mbar_init(&s.fac_full[i], 2);
      mbar_init(&s.fac_empty[i], kEpiWarps);
    }
    mbar_init(&s.drain, 1);
    fence_mbar_init();
  }
  grid_wait();
  if (warp == kEpiWarps) {
    build_tiles(p, kRows, s.tiles, lane);
  } else if (warp == kEpiWarps + 1) {
    tmem_alloc(&s.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  const int32_t tiles = s.tiles.first[p.E] * p.tiles_c;  // below 2^31: the host checks

  if (warp >= kEpiWarps) {
    setmaxnreg_dec<kOtherRegs>();
    if (warp == kEpiWarps) {
      // ---------------------------------------------------------- loads --
      const uint64_t pol = policy_evict_normal();
      const uint32_t done = smem_addr(s.done);
      uint32_t st = 0, use = 0;  // stage, its use
      bool ok = true;
      for (int32_t i = blockIdx.x; ok && i < tiles; i += gridDim.x) {
        const Tile t = tile_of(p, s.tiles, i, kRows, kCols, lane);
        const int32_t boxes = boxes_of(t);
        const uint32_t bytes = 2 * kWHalf + static_cast<uint32_t>(boxes) * (kBoxRows * kBlock);
        for (int32_t k = 0; k < p.inner; k += kBlock) {
          ok = mbar_wait_warp(done + st * 8, (use & 1) ^ 1u, wait_ns, p.err);
          if (!ok) break;
          if (elect_one()) {
            uint8_t* base = s.stage[st];
            uint64_t* bar = &s.full[st];
            s.cols[st] = min(kCols, p.outer - t.c0);
            mbar_arrive_expect_tx(bar, bytes);
            for (int h = 0; h < 2; ++h) {
              const int32_t c = t.c0 + h * kCols / 2;
              tma_load_3d(base + kABytes + h * kWHalf, &wmap, kT ? c : k, kT ? k : c, t.g, bar, pol);
            }
            if (boxes == kRows / kBoxRows)
              tma_load_2d(base, &amap, k, t.m0, bar, pol);
            else
              for (int b = 0; b < boxes; ++b)
                tma_load_2d(base + b * kBoxRows * kBlock, &amap32, k, t.m0 + b * kBoxRows, bar, pol);
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
      // ----------------------------------------------------------- MMAs --
      // One lane from here on, waits included: between the last release of an
      // accumulator and the next MMA there is little else to issue.
      if (elect_one()) {
        const uint32_t acc_empty = smem_addr(s.acc_empty), full = smem_addr(s.full);
        const uint32_t stage0 = smem_addr(s.stage);
        constexpr uint32_t wstep = kT ? (kSubK * kBlock) >> 4 : kSubK >> 4;
        uint32_t st = 0, st_use = 0, b = 0, use = 0;  // stage and accumulator, their uses
        bool ok = true, issued = false;
        for (int32_t i = blockIdx.x; ok && i < tiles; i += gridDim.x) {
          uint32_t idesc = 0;
          for (int32_t left = p.inner; left > 0; left -= kBlock) {
            // rows: K-major; weights: K-major rows of 128 bytes, or MN-major
            // (32 contraction rows = 4 KB, the column halves kWHalf apart)
            const uint32_t d = tmem + b * kCols, a0 = stage0 + st * kStageBytes;
            uint64_t ad = operand_desc_sw128(a0);
            uint64_t wd = operand_desc_sw128(a0 + kABytes, kWHalf);
            ok = mbar_wait_addr(full + st * 8, st_use & 1, wait_ns, p.err) &&
                 mbar_wait_addr(acc_empty + b * 8, (use & 1) ^ 1u, wait_ns, p.err);
            if (!ok) break;
            if (left == p.inner) {
              // the tile's columns: a multiple of 16, as the MMA's N has to be
              const uint32_t n = s.cols[st];
              // D fp32, e4m3 x e4m3, B MN-major if transposed, N = n, M = 128
              idesc = (1u << 4) | (kT ? 1u << 16 : 0u) | ((n >> 3) << 17) | (8u << 24);
            }
            tc_fence_after();
            tc_mma_e4m3<false>(d, ad, wd, idesc);
#pragma unroll
            for (int j = 1; j < kBlock / kSubK; ++j) {
              ad += kSubK >> 4;
              wd += wstep;
              if (j * kSubK < left) tc_mma_e4m3<true>(d, ad, wd, idesc);
            }
            tc_commit(&s.done[st]);
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
          tc_commit(&s.drain);
          mbar_wait_addr(smem_addr(&s.drain), 0, wait_ns, p.err);
        }
      }
      __syncwarp();
    } else {
      // -------------------------------------------------------- factors --
      // An entry's scales are loaded while the one before is worked on; only
      // rows that exist are read (clamped to one row, the loads of all blocks
      // would queue up at a single L2 line).
      const int32_t first = (warp - kEpiWarps - 2) * 64 + lane;
      float v[2][kScaleKb] = {}, w[2][kScaleKb];
      int32_t i = blockIdx.x, kb = 0;
      Tile t = {};
      auto load = [&]() {  // the entry (tile i, 128-blocks kb ..)
        if (kb == 0) t = tile_of(p, s.tiles, i, kRows, kCols, lane);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float* sb = p.sb + t.g * p.sb_expert +
                            static_cast<int64_t>(min(t.c0 / kBlock + h, p.sb_last)) * p.sb_c;
#pragma unroll
          for (int u = 0; u < kScaleKb; ++u)
            w[h][u] = __ldg(sb + static_cast<int64_t>(min(kb + u, p.kbs - 1)) * p.sb_k);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (first + 32 * j >= t.rows) continue;
          const float* sa = p.sa + static_cast<int64_t>(t.m0 + first + 32 * j) * p.kbs;
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
      uint32_t r = 0, use = 0;  // entry, its use
      bool ok = true;
      if (i < tiles) load();
      while (i < tiles) {
        ok = mbar_wait_warp(empty + r * 8, (use & 1) ^ 1u, wait_ns, p.err);
        if (!ok) break;
#pragma unroll
        for (int u = 0; u < kScaleKb; ++u) {
          const float w0 = rcp_approx(w[0][u]), w1 = rcp_approx(w[1][u]);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float ra = rcp_approx(v[j][u]);
            s.factor[r][u][0][first + 32 * j] = __fmul_rn(ra, w0);
            s.factor[r][u][1][first + 32 * j] = __fmul_rn(ra, w1);
          }
        }
        if (threadIdx.x == (kEpiWarps + 2) * 32) s.tile[r] = make_int4(t.m0, t.rows, t.c0, 0);
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.fac_full[r]);
        if (++r == kScaleRing) {
          r = 0;
          ++use;
        }
        kb += kScaleKb;
        if (kb >= p.kbs) {
          kb = 0;
          i += gridDim.x;
        }
        if (i < tiles) load();
      }
    }
  } else {
    // --------------------------------------------------------- epilogue --
    // Lane l of warp (q, hc) owns row 32 q + l of the tile and its columns
    // [128 hc, 128 hc + 128), one scale block of the weights.  A turn (one
    // 128-block) has to be short against the MMAs, and shared memory, which
    // carries their operands, answers slowly: a turn's factor is read, its
    // MMAs' completion probed and its first 32 columns loaded during the turn
    // before, and every load of TMEM runs under the multiply-adds of the
    // columns before it.  (All of a turn's loads at its start, to release the
    // accumulator sooner: 474 us instead of 463.)  The tile comes with its
    // factors: looking it up here took 1100 cycles, in which nothing moved.
    setmaxnreg_inc<kEpiRegs>();
    const int q = warp & 3, hc = warp >> 2;
    const uint32_t done = smem_addr(s.done), fac_full = smem_addr(s.fac_full);
    const uint32_t acc_empty = smem_addr(s.acc_empty);
    const uint32_t tmem0 = tmem + (static_cast<uint32_t>(32 * q) << 16) + hc * (kCols / 2);
    const uint32_t fac = smem_addr(&s.factor[0][0][hc][32 * q + lane]);
    const uint32_t tile = smem_addr(s.tile);
    constexpr uint32_t kFacKb = 2 * kRows * 4, kFacEntry = kScaleKb * kFacKb;
    uint32_t b = 0;               // accumulator
    uint32_t st = 0, use = 0;     // the stage whose MMAs filled it, its use
    uint32_t r = 0, fac_use = 0;  // entry of the factor ring, its use
    bool ready = false;           // the next MMAs are known to be complete
    bool hold = p.skip_arrival && blockIdx.x == 0;  // withhold the next release
    bool ok = true;
    for (int32_t i = blockIdx.x; ok && i < tiles; i += gridDim.x) {
      ok = mbar_wait_warp(fac_full + r * 8, fac_use & 1, wait_ns, p.err);
      if (!ok) break;
      const uint4 ti = lds128_ordered(tile + r * 16);
      float f = lds32_ordered(fac + r * kFacEntry);
      const int32_t row0 = static_cast<int32_t>(ti.x) + 32 * q;
      const int32_t rows = static_cast<int32_t>(ti.y) - 32 * q;  // of this warp, if positive
      const int32_t c = static_cast<int32_t>(ti.z) + hc * (kCols / 2);
      const bool mine = rows > 0 && c < p.outer;
      float acc[kChunks][kChunk];
#pragma unroll
      for (int a = 0; a < kChunks * kChunk; ++a) acc[a / kChunk][a % kChunk] = 0.0f;
      uint32_t e = 0;  // the 128-block's place in its entry
      uint32_t h0[kChunk], h1[kChunk];
      if (!__all_sync(0xffffffffu, ready)) {
        ok = mbar_wait_warp(done + st * 8, use & 1, wait_ns, p.err);
        if (!ok) break;
      }
      tc_fence_after();
      if (mine) {
        tmem_ld_32x32b_x32(tmem0 + b * kCols, h0);
        tmem_ld_wait32(h0);
      }
#pragma unroll 1
      for (int32_t left = p.kbs; left > 0; --left) {
        const uint32_t tacc = tmem0 + b * kCols;
        if (mine) {
          tmem_ld_32x32b_x32(tacc + kChunk, h1);
          scale_add(acc[0], h0, f);
          tmem_ld_wait32(h1);
          tmem_ld_32x32b_x32(tacc + 2 * kChunk, h0);
          scale_add(acc[1], h1, f);
          tmem_ld_wait32(h0);
          tmem_ld_32x32b_x32(tacc + 3 * kChunk, h1);
          scale_add(acc[2], h0, f);
          tmem_ld_wait32(h1);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && !hold) mbar_arrive_addr(acc_empty + b * 8);
        hold = false;
        b ^= 1;
        if (++st == kStages) {
          st = 0;
          ++use;
        }
        ready = mbar_test_addr(done + st * 8, use & 1);
        // on to the next 128-block's factor
        if (++e == kScaleKb || left == 1) {
          e = 0;
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.fac_empty[r]);
          if (++r == kScaleRing) {
            r = 0;
            ++fac_use;
          }
          if (left > 1) {
            ok = mbar_wait_warp(fac_full + r * 8, fac_use & 1, wait_ns, p.err);
            if (!ok) break;
          }
        }
        const float next = lds32_ordered(fac + r * kFacEntry + e * kFacKb);
        if (left > 1) {
          if (!__all_sync(0xffffffffu, ready)) {
            ok = mbar_wait_warp(done + st * 8, use & 1, wait_ns, p.err);
            if (!ok) break;
          }
          tc_fence_after();
          if (mine) {
            tmem_ld_32x32b_x32(tmem0 + b * kCols, h0);
            scale_add(acc[3], h1, f);
            tmem_ld_wait32(h0);
          }
        } else if (mine) {
          scale_add(acc[3], h1, f);
        }
        f = next;
      }
      if (!ok) break;
      if (!mine) continue;
      // 32 columns at a time: four lanes exchange their rows' 16-byte parts by
      // shuffles, so that a store covers 64-byte runs of eight rows.  (Staged in
      // shared memory: 456 us instead of 452; sent from there by TMA, with a
      // stage less for the operands, 480; without an exchange 495; exchanged by
      // pairs of lanes 472, by eight lanes 465 against 465 here.)
      const int part = lane & 3;
      uint16_t* orow = p.out + static_cast<int64_t>(row0 + (lane & ~3)) * p.outer + c + part * 8;
#pragma unroll
      for (int ch = 0; ch < kChunks; ++ch) {
        uint32_t x[4][4];  // [part][word] of this lane's row
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            x[w][j] = bf16x2_of(acc[ch][8 * w + 2 * j], acc[ch][8 * w + 2 * j + 1]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          swap_with<1>(x[0][j], x[1][j], lane);
          swap_with<1>(x[2][j], x[3][j], lane);
          swap_with<2>(x[0][j], x[2][j], lane);
          swap_with<2>(x[1][j], x[3][j], lane);
        }
        // x[k] is part lane & 3 of row (lane & ~3) + k
        const bool c_ok = c + ch * kChunk + part * 8 < p.outer;  // outer % 16 == 0
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if ((lane & ~3) + k < rows && c_ok)
            *reinterpret_cast<uint4*>(orow + static_cast<int64_t>(k) * p.outer + ch * kChunk) =
                make_uint4(x[k][0], x[k][1], x[k][2], x[k][3]);
      }
    }
    tc_fence_before();
  }

  __syncthreads();
  if (warp == kEpiWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Up to this many rows per group on average the kernel for few rows is ahead
// or close, whose narrower tiles spread the weights more evenly: in us, few /
// this, forward and transposed, at 16, 32, 48 and 96 rows each
//   64 experts of 2048 x 2048   43/49 44/50 47/51 54/54   43/47 44/48 46/49 54/52
//   16 of 4096 x 4096           48/49 50/50 52/50 56/52   46/44 47/45 49/46 54/47
//   8 of 8192 x 2048            25/27 26/27 28/28 33/29   22/31 23/32 25/32 28/33
//   8 of 2048 x 8192            22/32 23/33 25/34 28/34   25/26 26/26 28/27 33/28
// The rows are those of the buffer, also behind the last group's end.
constexpr int kFewRows = 48;

}  // namespace

gq_status setup(DeviceInfo& info) {
  for (const void* f : {reinterpret_cast<const void*>(product_kernel<false>),
                        reinterpret_cast<const void*>(product_kernel<true>)}) {
    gq_status st = check_cuda(
        cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmemBytes)),
        "grouped_mm: shared memory size");
    if (st != GQ_OK) return st;
    // a split above the launch's registers would wait for ever
    cudaFuncAttributes a;
    st = check_cuda(cudaFuncGetAttributes(&a, f), "grouped_mm: registers");
    if (st != GQ_OK) return st;
    if (a.numRegs * kThreads < 32 * (kEpiWarps * kEpiRegs + (kThreads / 32 - kEpiWarps) * kOtherRegs))
      return fail(GQ_ERR_UNSUPPORTED, "grouped_mm: built with %d registers per thread", a.numRegs);
  }
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

  const int64_t most = (M / kRows + (E < M ? E : M)) * p.tiles_c;  // tiles of any offsets
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
  const unsigned grid = static_cast<unsigned>(most < info.sm_count ? most : info.sm_count);
  const auto kernel = transposed ? product_kernel<true> : product_kernel<false>;
  return launch_chained("grouped_mm: launch", kernel, dim3(grid), kThreads, kSmemBytes, stream, 1,
                        amap, amap32, wmap, p);
}

}  // namespace gmm
}  // namespace gq
