// gq_grouped_mm.cu -- the grouped products of block-quantized rows with
// block-quantized stacked weights, one expert per token group, on the
// sm_103a tensor cores (tcgen05, TMEM accumulators, TMA operands):
//   forward     out[m][n] = sum_k A[m][k] * W[e][n][k]
//   transposed  out[m][k] = sum_n A[m][n] * W[e][n][k]
//   gated       h[m][n] = act(sum_k A[m][k] W[e][0][n][k]) * sum_k A[m][k] W[e][1][n][k]
//   gated grad  out[m][k] = sum_n A[m][0][n] W[e][0][n][k] + A[m][1][n] W[e][1][n][k]
// with A = qa / sa (one scale per row and 128 contraction columns) and
// W = qb / sb (one scale per 128x128 block).  Within a 128-block kb of the
// contraction both scales are constant for a row m and 128 output columns c,
//   out[m][c] = sum_kb ( 1/sa[m][kb] * 1/sb[e][c/128, kb] ) * P_kb[m][c],
// P_kb the plain sum of the block's e4m3 products.  The tensor cores form
// P_kb in TMEM (fp32); the epilogue warps read it, multiply by the factor
// and add it to fp32 accumulators in registers, rounded once.  The gated
// tile is 128 columns of both projections, so that activation, product and
// the 1x128 quantization need nothing but the tile.
//
// A block takes tiles of 128 rows x 256 output columns, 128 contraction
// columns at a time.  The rows are the MMA's M operand, so that a TMEM lane
// is a row and its factor one register: with the weights as M a lane would
// need every row's factor, and those loads alone -- shared memory returns 128
// bytes a cycle -- would cost as much as the MMAs.
//
// What bounds it, 16,640 rows in 16 groups (16 matrices of 8192 x 4096):
// * a long run, the power limit: the clock falls to 1.5 GHz where it is 1.8 for
//   a single call.  grad_input of the gated block 480 to 515 us (2.2 to 2.3
//   PFLOP/s), by the card; where it took 506, 418 were left without
//   multiply-adds, TMEM loads and stores;
// * one call, 811 cycles a 128-block, 455 us: the MMAs are 512 and the operands
//   770, 48 KB at the 64 bytes a cycle that L2 delivers to an SM.  A pair of
//   blocks (cta_group::2) loads 32 KB per block, but its accumulators are
//   released across blocks, and with two of them, all of TMEM, that round trip
//   (1100 cycles: release, first MMA, completion, wake-up) takes the place of the
//   loads: 860 cycles, and a group is padded to 256 rows.  Halves of the
//   accumulators released apart (MMAs of N = 128): the same 460 and 490 us;
//   two issuing warps, three barriers probed ahead: no faster;
// * rows that are not whole lines, pairs of blocks (see kPairRows): 24,500 live
//   rows of 40 experts, 1360 x 2064, gated to fp8: 264 us alone, 163 to 190 in
//   pairs.
// The gated form adds 3500 cycles a tile for the stores of 112 KB (both rows
// and projections, 32 bytes a cycle) and 1600 for the activation: 16 x 2 x 4096 x
// 4096, everything written: 525 us, in a long run 545 to 570; the plain product
// with the same matrices 467 and 490 to 530.
//
// One persistent block per SM -- or, where the gated forms have few tiles, a cluster
// per tile (see Split and kSplitKbs) -- whose warps are:
//   0-7   epilogue: lane quarter w % 4 (32 rows), column half w / 4 (gated: 64
//         columns of both projections);
//   8     TMA loads (one lane);
//   9     TMEM allocation and the MMAs (one lane, of a pair the first block's);
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

constexpr int kRows = 128;        // rows of a tile, per block
constexpr int kCols = 256;        // output columns of a tile
constexpr int kBoxRows = 32;      // rows per TMA box where a tile has few
constexpr int kABytes = kRows * kBlock;      // 16 KB
constexpr int kWHalf = kCols / 2 * kBlock;   // 16 KB: half of the output columns
constexpr int kBufs = 2;          // accumulators in TMEM
constexpr uint32_t kTmemCols = kBufs * kCols;
constexpr int kEpiWarps = 8;      // two per TMEM lane quarter
constexpr int kThreads = (kEpiWarps + 4) * 32;
constexpr int kEpiRegs = 232;     // registers per thread after the split:
constexpr int kOtherRegs = 40;    // what the block was launched with, no more
constexpr int kChunk = 32;        // columns per step of the epilogue
constexpr int kChunks = kCols / 2 / kChunk;
constexpr int kScaleRing = 2;
constexpr int kMostParts = 4;     // blocks that share a tile's contraction, at most
static_assert(kTmemCols == 512 && kChunks == 4, "two accumulators fill the TMEM");

// Blocks that share a tile: one, with all of its output columns' weights, or
// two (a pair, cta_group::2), each with half of them.
template <int kBlocks>
struct Smem {
  static constexpr int kStages = kBlocks == 2 ? 6 : 4;
  static constexpr int kStageBytes = kABytes + 2 / kBlocks * kWHalf;
  uint8_t stage[kStages][kStageBytes];  // 1024-byte aligned (swizzle atoms)
  float factor[kScaleRing][kScaleKb][2][kRows];  // of the tile's two column halves
  int4 tile[kScaleRing];         // the entry's tile: first row and rows of this block, first column
  int32_t cols[kStages];         // mma_cols of the stage's tile
  TileTable tiles;
  uint64_t full[kStages];         // the stage's loads in every block (the first block)
  uint64_t done[kStages];         // its MMAs are complete: the stage is free, the accumulator full
  uint64_t acc_empty[kBufs];      // accumulator read (8 warps of every block; the first block)
  uint64_t fac_full[kScaleRing];  // factors written (2 warps)
  uint64_t fac_empty[kScaleRing]; // factors read (8 warps)
  uint64_t drain;
  uint64_t share[4];              // kGated: both halves of a row have their maximum (2 warps)
  float most[2][2][kRows];        // kGated: those maxima, by tile parity and half
  uint32_t tmem_base;
};
template <int kBlocks>
constexpr size_t smem_bytes() {
  static_assert(sizeof(Smem<kBlocks>) + 1024 <= 227 * 1024, "fits one SM's shared memory");
  return sizeof(Smem<kBlocks>) + 1024;
}

// The tensor-core and TMA instructions for a block alone or in a pair.  `bar`
// and acc_empty of a pair are the first block's, as shared::cluster addresses.
template <int kBlocks>
struct Group;

template <>
struct Group<1> {
  static __device__ __forceinline__ uint32_t of_first(uint32_t addr) { return addr; }
  static __device__ __forceinline__ void alloc(uint32_t* dst) {
    tmem_alloc(dst, kTmemCols);
    tmem_relinquish();
  }
  static __device__ __forceinline__ void dealloc(uint32_t addr) { tmem_dealloc(addr, kTmemCols); }
  static __device__ __forceinline__ void load_2d(void* dst, const CUtensorMap* map, int32_t x,
                                                 int32_t y, uint32_t bar, uint64_t pol) {
    tma_load_2d_addr(dst, map, x, y, bar, pol);
  }
  static __device__ __forceinline__ void load_3d(void* dst, const CUtensorMap* map, int32_t x,
                                                 int32_t y, int32_t z, uint32_t bar, uint64_t pol) {
    tma_load_3d_addr(dst, map, x, y, z, bar, pol);
  }
  template <bool kAccumulate>
  static __device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
    tc_mma_e4m3<kAccumulate>(d, a, b, idesc);
  }
  static __device__ __forceinline__ void commit(uint64_t* bar) { tc_commit(bar); }
  static __device__ __forceinline__ void commit_first(uint64_t* bar) { tc_commit(bar); }
  static __device__ __forceinline__ void release(uint32_t bar) { mbar_arrive_addr(bar); }
  static __device__ __forceinline__ void sync() {}
};

template <>
struct Group<2> {
  static __device__ __forceinline__ uint32_t of_first(uint32_t addr) { return map_cluster(addr, 0); }
  static __device__ __forceinline__ void alloc(uint32_t* dst) {
    tmem_alloc_pair(dst, kTmemCols);
    tmem_relinquish_pair();
  }
  static __device__ __forceinline__ void dealloc(uint32_t addr) { tmem_dealloc_pair(addr, kTmemCols); }
  static __device__ __forceinline__ void load_2d(void* dst, const CUtensorMap* map, int32_t x,
                                                 int32_t y, uint32_t bar, uint64_t pol) {
    tma_load_2d_pair(dst, map, x, y, bar, pol);
  }
  static __device__ __forceinline__ void load_3d(void* dst, const CUtensorMap* map, int32_t x,
                                                 int32_t y, int32_t z, uint32_t bar, uint64_t pol) {
    tma_load_3d_pair(dst, map, x, y, z, bar, pol);
  }
  template <bool kAccumulate>
  static __device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
    tc_mma_e4m3_pair<kAccumulate>(d, a, b, idesc);
  }
  static __device__ __forceinline__ void commit(uint64_t* bar) { tc_commit_pair(bar, 3); }
  static __device__ __forceinline__ void commit_first(uint64_t* bar) { tc_commit_pair(bar, 1); }
  static __device__ __forceinline__ void release(uint32_t bar) { mbar_arrive_cluster(bar); }
  static __device__ __forceinline__ void sync() {
    cluster_arrive();
    cluster_wait();
  }
};

// TMA boxes of kBoxRows rows for a block's rows (4: one box of kRows).
__device__ __forceinline__ int32_t boxes_of(int32_t rows) {
  return (max(min(rows, kRows), 0) + kBoxRows - 1) / kBoxRows;
}

// The MMA's N for a tile: its output columns, of a pair in equal halves of whole
// 16s; kGated: 128 of each projection, what lies behind the last reads zeros.
template <int kForm, int kBlocks>
__device__ __forceinline__ int32_t mma_cols(const Params& p, int32_t c0) {
  const int32_t left = p.outer - c0;
  if (kForm == kGated || left >= kCols) return kCols;
  return kBlocks == 2 ? (left + 31) / 32 * 32 : left;
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

// Stores 64 bytes of each of this warp's rows, `out` pointing at this lane's part
// of them in row (lane & ~3): four lanes exchange their
// rows' 16-byte parts by shuffles, so that a store covers 64-byte runs of eight
// rows.  (Staged in shared memory: 456 us instead of 452; sent from there by
// TMA, with a stage less for the operands, 480; without an exchange 495;
// exchanged by pairs of lanes 472, by eight lanes 465 against 465 here.)
__device__ __forceinline__ void store_parts(uint32_t (&x)[4][4], uint8_t* out, int64_t pitch_bytes,
                                            int32_t rows, bool c_ok, int lane) {
  // x[part][word] of this lane's row
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    swap_with<1>(x[0][j], x[1][j], lane);
    swap_with<1>(x[2][j], x[3][j], lane);
    swap_with<2>(x[0][j], x[2][j], lane);
    swap_with<2>(x[1][j], x[3][j], lane);
  }
  // x[k] is part lane & 3 of row (lane & ~3) + k
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if ((lane & ~3) + k < rows && c_ok)
      *reinterpret_cast<uint4*>(out + k * pitch_bytes) = make_uint4(x[k][0], x[k][1], x[k][2], x[k][3]);
}

__device__ __forceinline__ void store_bf16(const float (&v)[kChunk], uint16_t* out, int64_t pitch,
                                           int32_t rows, bool c_ok, int lane) {
  uint32_t x[4][4];
#pragma unroll
  for (int w = 0; w < 4; ++w)
#pragma unroll
    for (int j = 0; j < 4; ++j) x[w][j] = bf16x2_of(v[8 * w + 2 * j], v[8 * w + 2 * j + 1]);
  store_parts(x, reinterpret_cast<uint8_t*>(out), pitch * 2, rows, c_ok, lane);
}

template <int kForm, int kBlocks, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap amap,
                   const __grid_constant__ CUtensorMap amap32,
                   const __grid_constant__ CUtensorMap wmap, const Params p) {
  // aligned by an offset, so that the compiler still knows the address space
  constexpr bool kT = is_transposed(kForm);
  // output columns of a tile; kGated: as many of each projection
  constexpr int kTileCols = kForm == kGated ? kCols / 2 : kCols;
  constexpr int kTileRows = kBlocks * kRows;
  using G = Group<kBlocks>;
  constexpr int kStages = Smem<kBlocks>::kStages, kStageBytes = Smem<kBlocks>::kStageBytes;
  extern __shared__ uint8_t smem_raw[];
  Smem<kBlocks>& s = *reinterpret_cast<Smem<kBlocks>*>(smem_raw + (-smem_addr(smem_raw) & 1023u));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  static_assert(kBlocks == 1 || !kSplit, "a cluster is a pair or shares a contraction");
  const int32_t rank = kBlocks == 2 ? static_cast<int32_t>(cluster_rank()) : 0;
  const Split part = split_of<kSplit>(p);
  const int32_t sharing = kBlocks * part.parts;
  const int32_t groups = gridDim.x / sharing, group = blockIdx.x / sharing;
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
    for (int b = 0; b < kBufs; ++b) mbar_init(&s.acc_empty[b], kBlocks * kEpiWarps);
    for (int i = 0; i < kScaleRing; ++i) {
      mbar_init(&s.fac_full[i], 2);
      mbar_init(&s.fac_empty[i], kEpiWarps);
    }
    mbar_init(&s.drain, 1);
    for (int i = 0; i < 4; ++i) mbar_init(&s.share[i], 2);
    fence_mbar_init();
  }
  grid_wait();
  if (may_choose(kForm) && p.pairs_only != 0) {
    bool past = false;
    for (int32_t g = threadIdx.x; g < p.E; g += kThreads) past |= __ldg(p.offs + g) > p.pairs_over;
    if ((__syncthreads_or(past) != 0) != (p.pairs_only > 0)) return;
  }
  if (warp == kEpiWarps) {
    build_tiles(p, kTileRows, s.tiles, lane);
  } else if (warp == kEpiWarps + 1) {
    G::alloc(&s.tmem_base);
  }
  tc_fence_before();
  __syncthreads();
  G::sync();  // the other block's barriers are ready as well
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  const int32_t tiles = s.tiles.first[p.E] * p.tiles_c;  // below 2^31: the host checks

  bool joined = false;  // split: this warp has met the cluster's barrier
  if (warp >= kEpiWarps) {
    setmaxnreg_dec<kOtherRegs>();
    if (warp == kEpiWarps) {
      // ---------------------------------------------------------- loads --
      const uint64_t pol = policy_evict_normal();
      const uint32_t done = smem_addr(s.done), full = G::of_first(smem_addr(s.full));
      uint32_t st = 0, use = 0;  // stage, its use
      bool ok = true;
      for (int32_t i = group; ok && i < tiles; i += groups) {
        const Tile t = tile_of(p, s.tiles, i, kTileRows, kTileCols, lane);
        const int32_t boxes = boxes_of(t.rows - rank * kRows), m0 = t.m0 + rank * kRows;
        const int32_t cols = mma_cols<kForm, kBlocks>(p, t.c0);
        int32_t rows32 = boxes;  // of all blocks
        if (kBlocks == 2) rows32 = boxes_of(t.rows) + boxes_of(t.rows - kRows);
        const uint32_t bytes = 2 * kWHalf + static_cast<uint32_t>(rows32) * (kBoxRows * kBlock);
        for (int32_t kb = part.kb0; kb < part.kb1; ++kb) {
          const int32_t k = column_of<kForm>(p, kb), half = half_of<kForm>(p, kb);
          ok = mbar_wait_warp(done + st * 8, (use & 1) ^ 1u, wait_ns, p.err);
          if (!ok) break;
          if (elect_one()) {
            uint8_t* base = s.stage[st];
            const uint32_t bar = full + st * 8;
            if (rank == 0) {  // the bytes of every block complete on the first one's barrier
              s.cols[st] = cols;
              mbar_arrive_expect_tx(&s.full[st], bytes);
            }
#pragma unroll
            for (int j = 0; j < 2 / kBlocks; ++j) {
              const int32_t h = kBlocks == 2 ? rank : j;  // which half of the columns
              const int32_t c = kForm == kGated ? t.c0 : t.c0 + h * (kBlocks == 2 ? cols / 2 : kCols / 2);
              const int32_t w = kForm == kGated ? 2 * t.g + h : kForm == kGatedGrad ? 2 * t.g + half : t.g;
              G::load_3d(base + kABytes + j * kWHalf, &wmap, kT ? c : k, kT ? k : c, w, bar, pol);
            }
            auto load_rows = [&](const CUtensorMap* map, int32_t row) {
              uint8_t* const to = base + row * kBlock;
              if (kForm == kGatedGrad)
                G::load_3d(to, map, k, half, m0 + row, bar, pol);
              else
                G::load_2d(to, map, k, m0 + row, bar, pol);
            };
            if (boxes == kRows / kBoxRows)
              load_rows(&amap, 0);
            else
              for (int b = 0; b < boxes; ++b) load_rows(&amap32, b * kBoxRows);
          }
          __syncwarp();
          if (++st == kStages) {
            st = 0;
            ++use;
          }
        }
      }
      // neither block may exit while a load is still writing its memory, also
      // after a wait that ran out; the MMAs that read it are waited for below
      for (uint32_t u = 0; rank == 0 && u < kStages; ++u) {
        const uint32_t uses = use + (u < st ? 1 : 0);
        if (uses > 0) mbar_wait_warp(smem_addr(&s.full[u]), (uses - 1) & 1, wait_ns, p.err);
      }
    } else if (warp == kEpiWarps + 1) {
      // ----------------------------------------------------------- MMAs --
      // One lane of the first block from here on, waits included: between the
      // last release of an accumulator and the next MMA there is little else to
      // issue.
      if (rank == 0 && elect_one()) {
        const uint32_t acc_empty = smem_addr(s.acc_empty), full = smem_addr(s.full);
        const uint32_t stage0 = smem_addr(s.stage);
        constexpr uint32_t wstep = kT ? (kSubK * kBlock) >> 4 : kSubK >> 4;
        uint32_t st = 0, st_use = 0, b = 0, use = 0;  // stage and accumulator, their uses
        bool ok = true, issued = false;
        for (int32_t i = group; ok && i < tiles; i += groups) {
          uint32_t idesc = 0;
          for (int32_t kb = part.kb0; kb < part.kb1; ++kb) {
            const int32_t left = p.inner - column_of<kForm>(p, kb);
            // rows: K-major; weights: K-major rows of 128 bytes, or MN-major
            // (32 contraction rows = 4 KB, one block's halves of the columns kWHalf apart)
            const uint32_t d = tmem + b * kCols, a0 = stage0 + st * kStageBytes;
            const uint64_t ad = operand_desc_sw128(a0), wd = operand_desc_sw128(a0 + kABytes, kWHalf);
            ok = mbar_wait_addr(full + st * 8, st_use & 1, wait_ns, p.err) &&
                 mbar_wait_addr(acc_empty + b * 8, (use & 1) ^ 1u, wait_ns, p.err);
            if (!ok) break;
            if (kb == part.kb0)  // D fp32, e4m3 x e4m3, B MN-major if transposed, N, M
              idesc = (1u << 4) | (kT ? 1u << 16 : 0u) | (static_cast<uint32_t>(kTileRows >> 4) << 24) |
                      ((static_cast<uint32_t>(s.cols[st]) >> 3) << 17);
            tc_fence_after();
            G::template mma<false>(d, ad, wd, idesc);
            if (left >= kBlock) {
#pragma unroll
              for (int j = 1; j < kBlock / kSubK; ++j)
                G::template mma<true>(d, ad + j * (kSubK >> 4), wd + j * wstep, idesc);
            } else {
#pragma unroll 1
              for (int j = 1; j * kSubK < left; ++j)
                G::template mma<true>(d, ad + j * (kSubK >> 4), wd + j * wstep, idesc);
            }
            G::commit(&s.done[st]);
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
          G::commit_first(&s.drain);
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
      float v[2][kScaleKb] = {}, ws[2][kScaleKb];
      int32_t i = group, kb = part.kb0;
      Tile t = {};
      auto load = [&]() {  // the entry (tile i, 128-blocks kb ..)
        if (kb == part.kb0) {
          t = tile_of(p, s.tiles, i, kTileRows, kTileCols, lane);
          t.m0 += rank * kRows;
          t.rows -= rank * kRows;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int32_t w = kForm == kGated ? 2 * t.g + h : t.g;
          const int32_t c = kForm == kGated ? t.c0 / kBlock : min(t.c0 / kBlock + h, p.sb_last);
          const float* sb = p.sb + w * p.sb_expert + static_cast<int64_t>(c) * p.sb_c;
#pragma unroll
          for (int u = 0; u < kScaleKb; ++u)
            ws[h][u] = __ldg(sb + static_cast<int64_t>(min(kb + u, p.kbs - 1)) * p.sb_k);
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
          const float w0 = rcp_approx(ws[0][u]), w1 = rcp_approx(ws[1][u]);
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
        if (kb >= part.kb1) {
          kb = part.kb0;
          i += groups;
        }
        if (i < tiles) load();
      }
    }
  } else {
    // --------------------------------------------------------- epilogue --
    // Lane l of warp (q, hc) owns row 32 q + l of the tile and its columns
    // [128 hc, 128 hc + 128), one scale block of the weights (kGated: [64 hc,
    // 64 hc + 64) of both projections, one factor for each).  A turn (one
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
    const uint32_t acc_empty = G::of_first(smem_addr(s.acc_empty));
    constexpr int kMine = kTileCols / 2;  // output columns of this warp
    const uint32_t tmem0 = tmem + (static_cast<uint32_t>(32 * q) << 16) + hc * kMine;
    // where this warp's chunk ch begins in an accumulator
    auto col = [](int ch) {
      return kForm == kGated ? (ch >> 1) * kTileCols + (ch & 1) * kChunk : ch * kChunk;
    };
    const uint32_t fac = smem_addr(&s.factor[0][0][kForm == kGated ? 0 : hc][32 * q + lane]);
    const uint32_t tile = smem_addr(s.tile);
    constexpr uint32_t kFacKb = 2 * kRows * 4, kFacEntry = kScaleKb * kFacKb;
    uint32_t b = 0;               // accumulator
    uint32_t st = 0, use = 0;     // the stage whose MMAs filled it, its use
    uint32_t r = 0, fac_use = 0;  // entry of the factor ring, its use
    bool ready = false;           // the next MMAs are known to be complete
    uint32_t shares = 0;          // exchanges with the other half's warp so far
    bool hold = p.skip_arrival && blockIdx.x == 0;  // withhold the next release
    bool ok = true;
    for (int32_t i = group; ok && i < tiles; i += groups) {
      ok = mbar_wait_warp(fac_full + r * 8, fac_use & 1, wait_ns, p.err);
      if (!ok) break;
      const uint4 ti = lds128_ordered(tile + r * 16);
      float f = lds32_ordered(fac + r * kFacEntry), f1 = f;  // kGated: f1 is the up projection's
      if (kForm == kGated) f1 = lds32_ordered(fac + r * kFacEntry + kRows * 4);
      const int32_t row0 = static_cast<int32_t>(ti.x) + 32 * q;
      const int32_t rows = static_cast<int32_t>(ti.y) - 32 * q;  // of this warp, if positive
      const int32_t c = static_cast<int32_t>(ti.z) + hc * kMine;
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
      for (int32_t left = part.kb1 - part.kb0; left > 0; --left) {
        const uint32_t tacc = tmem0 + b * kCols;
        if (mine) {
          tmem_ld_32x32b_x32(tacc + col(1), h1);
          scale_add(acc[0], h0, f);
          tmem_ld_wait32(h1);
          tmem_ld_32x32b_x32(tacc + col(2), h0);
          scale_add(acc[1], h1, f);
          tmem_ld_wait32(h0);
          tmem_ld_32x32b_x32(tacc + col(3), h1);
          scale_add(acc[2], h0, kForm == kGated ? f1 : f);
          tmem_ld_wait32(h1);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && !hold) G::release(acc_empty + b * 8);
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
        float next1 = next;
        if (kForm == kGated) next1 = lds32_ordered(fac + r * kFacEntry + e * kFacKb + kRows * 4);
        if (left > 1) {
          if (!__all_sync(0xffffffffu, ready)) {
            ok = mbar_wait_warp(done + st * 8, use & 1, wait_ns, p.err);
            if (!ok) break;
          }
          tc_fence_after();
          if (mine) {
            tmem_ld_32x32b_x32(tmem0 + b * kCols, h0);
            scale_add(acc[3], h1, kForm == kGated ? f1 : f);
            tmem_ld_wait32(h0);
          }
        } else if (mine) {
          scale_add(acc[3], h1, kForm == kGated ? f1 : f);
        }
        f = next;
        f1 = next1;
      }
      if (!ok) break;
      if (!mine) continue;
      if constexpr (kSplit) {
        // the stages are free: all MMAs of the block are complete
        const uint32_t own = smem_addr(s.stage) + (warp * (kChunks * kChunk / 4) * 32 + lane) * 16;
        if (!part.mine(q)) {
#pragma unroll
          for (int k = 0; k < kChunks * kChunk; k += 4) {
            const float* v = &acc[k / kChunk][k % kChunk];
            sts128(own + k / 4 * 512, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]),
                                                 __float_as_uint(v[2]), __float_as_uint(v[3])));
          }
        }
        cluster_arrive();
        cluster_wait();
        joined = true;
        if (!part.mine(q)) continue;
        // (a0 + a1) + (a2 + a3), a_i the sums of block i: each addition commutes, so that
        // a row has the same bits whichever block adds it up, wherever in the tile it
        // is.  Eight words are under way at a time.
        static_assert(kMostParts <= 4, "two rounds of pairs");
        const uint32_t other = map_cluster(own, part.rank ^ 1);
#pragma unroll
        for (int k0 = 0; k0 < kChunks * kChunk; k0 += 32) {
          uint4 v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = ld_cluster_128(other + (k0 / 4 + k) * 512);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float* const o = &acc[k0 / kChunk][4 * k];
            o[0] += __uint_as_float(v[k].x);
            o[1] += __uint_as_float(v[k].y);
            o[2] += __uint_as_float(v[k].z);
            o[3] += __uint_as_float(v[k].w);
          }
        }
        if (part.parts > 2) {
          const uint32_t two = map_cluster(own, part.rank ^ 2), three = map_cluster(own, part.rank ^ 3);
#pragma unroll
          for (int k0 = 0; k0 < kChunks * kChunk; k0 += 16) {
            uint4 v[4], w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              v[k] = ld_cluster_128(two + (k0 / 4 + k) * 512);
              w[k] = ld_cluster_128(three + (k0 / 4 + k) * 512);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float* const o = &acc[k0 / kChunk][k0 % kChunk + 4 * k];
              o[0] += __uint_as_float(v[k].x) + __uint_as_float(w[k].x);
              o[1] += __uint_as_float(v[k].y) + __uint_as_float(w[k].y);
              o[2] += __uint_as_float(v[k].z) + __uint_as_float(w[k].z);
              o[3] += __uint_as_float(v[k].w) + __uint_as_float(w[k].w);
            }
          }
        }
      }
      const int col8 = lane & 3;
      const int64_t row = row0 + (lane & ~3);
      if constexpr (kForm != kGated) {
        uint16_t* const orow = p.out + row * p.outer + c + col8 * 8;
#pragma unroll
        for (int ch = 0; ch < kChunks; ++ch)
          store_bf16(acc[ch], orow + ch * kChunk, p.outer, rows,
                     c + ch * kChunk + col8 * 8 < p.outer, lane);  // outer % 16 == 0
      } else {
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          const int32_t at = c + ch * kChunk + col8 * 8;
          const bool in = at < p.outer;  // outer % 16 == 0
          if (p.pre != nullptr) {  // the projections, as they are
            uint16_t* const prow = p.pre + row * 2 * p.outer + at;
            store_bf16(acc[ch], prow, 2 * static_cast<int64_t>(p.outer), rows, in, lane);
            store_bf16(acc[ch + 2], prow + p.outer, 2 * static_cast<int64_t>(p.outer), rows, in, lane);
          }
          gated::gate(p.act, acc[ch], acc[ch + 2]);
          if (p.out != nullptr) store_bf16(acc[ch], p.out + row * p.outer + at, p.outer, rows, in, lane);
        }
        if (p.q == nullptr) continue;
        // a 1x128 block is this warp's row and that of the warp of the other half
        // of the columns: they exchange their maxima (a NaN does not count; columns
        // past the last are zeros)
        float most = 0.0f;
#pragma unroll
        for (int ch = 0; ch < 2; ++ch)
#pragma unroll
          for (int j = 0; j < kChunk; ++j) most = fmaxf(most, fabsf(acc[ch][j]));
        if (static_cast<int32_t>(ti.z) + kMine < p.outer) {
          const uint32_t buf = smem_addr(&s.most[shares & 1][0][32 * q + lane]);
          sts32(buf + hc * kRows * 4, most);
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.share[q]);
          ok = mbar_wait_warp(smem_addr(&s.share[q]), shares & 1, wait_ns, p.err);
          if (!ok) break;
          ++shares;
          most = fmaxf(most, lds32_ordered(buf + (hc ^ 1) * kRows * 4));
        }
        const float sc = scale_from_amax_bits(__float_as_uint(most), p.pow2);
        uint32_t x[4][4];
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float* v = &acc[w >> 1][(w & 1) * 16 + 4 * j];
            x[w][j] = quant4f(make_float4(v[0], v[1], v[2], v[3]), sc);
          }
        store_parts(x, p.q + row * p.outer + c + col8 * 16, p.outer, rows, c + col8 * 16 < p.outer, lane);
        if (hc == 0 && lane < rows)
          p.scales[static_cast<int64_t>(row0 + lane) * ((p.outer + kBlock - 1) / kBlock) + c / kBlock] = sc;
      }
    }
    tc_fence_before();
  }
  if (kSplit) {
    // Every thread meets the cluster's barrier twice: with the sums written, and
    // with them read, before a block that holds some may leave.
    if (!joined) {
      cluster_arrive();
      cluster_wait();
    }
    cluster_arrive();
    cluster_wait();
  }

  __syncthreads();
  G::sync();  // neither block leaves while the other may still signal it
  if (warp == kEpiWarps + 1) {
    tc_fence_after();
    G::dealloc(tmem);
  }
}

// Up to this many rows per group on average the kernel for few rows is ahead
// or close, whose narrower tiles spread the weights more evenly: in us, few /
// this, forward and transposed, at 16, 32, 48 and 96 rows each
//   64 experts of 2048 x 2048   43/49 44/50 47/51 54/54   43/47 44/48 46/49 54/52
//   16 of 4096 x 4096           48/49 50/50 52/50 56/52   46/44 47/45 49/46 54/47
//   8 of 8192 x 2048            25/27 26/27 28/28 33/29   22/31 23/32 25/32 28/33
//   8 of 2048 x 8192            22/32 23/33 25/34 28/34   25/26 26/26 28/27 33/28
// The gated form has half as many rows in a tile there: fp8 rows, at 16, 24, 32 and 48
//   64 pairs of 1024 x 2048     48/49 47/49 47/50 52/49
//   64 of 1424 x 2064           66/69 68/71 70/72 77/78, all outputs 73/73 78/75 85/78 96/86
//   16 of 2048 x 4096           45/48 47/48 47/49 54/49
//   8 of 768 x 2048             11/11 13/12 14/12 13/12
//   one of 2048 x 4096          9.9/11.6 11.6/11.6 12.1/11.6 14.0/11.8
// The rows are those of the buffer, also behind the last group's end; so are the
// tiles by which parts_of shares them out.
constexpr int kFewRows = 48, kFewRowsGated = 24;

// Block pairs where rows of an operand begin anywhere in a 128-byte line (their
// length is no multiple of 64 bytes): nearly each 128 bytes of a box are then two
// lines for L2, and the operands' arrival binds; a pair has each line of the weights
// loaded once for both blocks.  But it pads groups to 256 rows, so not for few,
// nor where there are few tiles to share out.  In us, pairs / single blocks, uneven
// groups of 64, 96, 128, 192 and 512 rows of 64 experts, 1424 x 2064:
//   gated 102/85 105/103 109/116 134/156 251/342
//   grad_input of it 93/86 97/107 114/126 138/162 280/375
//   forward 92/85 97/105 103/121 130/159 274/354, transposed 90/78 92/96 104/113 118/144 234/330
// With rows of whole lines (64 of 1024 x 2048, gated): 64/51 64/57 71/57 86/71
// (200 rows) 127/120 (400), at 1040 rows of 16 x 2048 x 4096 232/238.
// For the plain products the rows are those in front of the last end.  The host knows
// the buffer's alone, of which a layer with a part of the experts may fill little:
// where these are enough for pairs, it launches both kernels, and the blocks of the
// one that the ends do not want leave again: 1.5 us in a call, up to 4 % where the
// groups have many rows.  64 groups as above in a buffer of 16 times their rows, at 16,
// 32 and 64 rows each, pairs / single blocks / both launched
//   forward 50/39/40 51/40/42 54/45/47, transposed 49/41/42 50/42/42 53/47/48
// The gated forms go by the buffer's rows: gated 99/73/79 98/74/82 101/79/87 there,
// grad_input of it 84/75/75 86/79/79 90/86/87, but 40 groups of 614 rows in a buffer of
// four times as many, gated to fp8, 186/-/190 in a run of nothing but this call.
constexpr int kPairRows = 96;
constexpr int kPairTiles = 3;  // per SM

// Blocks share a tile of the gated forms where there are few tiles and more than
// this many 128-blocks: joining the sums takes 4 us, a 128-block 0.45.  In us, one
// block / as many as parts_of gives, 128-blocks in brackets: 128 rows of one
// expert, 2 x 2048 x 4096, gated 17.3/13.7 (32), its grad_input 16.8/12.2 (32); 100 of
// one, 2 x 768 x 7168, 25.6/16.1 (56) and 9.1/11.1 (12); 256 of four, 2 x 1024 x 4096,
// 17.3/15.3 (32); 128 of two, 2 x 1408 x 2048, 11.3/12.1 (16) and 12.8/12.1 (22).
// (Each block's own sum first, whichever it is, 0.7 us less where four share a tile;
// but then a row's last bits go by its place in the tile.)
constexpr int kSplitKbs = 20;

}  // namespace

namespace {

template <int kForm, int kBlocks, bool kSplit>
gq_status setup_kernel() {
  const auto kernel = product_kernel<kForm, kBlocks, kSplit>;
  gq_status st = check_cuda(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(smem_bytes<kBlocks>())),
                            "grouped_mm: shared memory size");
  if (st != GQ_OK) return st;
  // a split above the launch's registers would wait for ever
  cudaFuncAttributes a;
  st = check_cuda(cudaFuncGetAttributes(&a, kernel), "grouped_mm: registers");
  if (st != GQ_OK) return st;
  if (a.numRegs * kThreads < 32 * (kEpiWarps * kEpiRegs + (kThreads / 32 - kEpiWarps) * kOtherRegs))
    return fail(GQ_ERR_UNSUPPORTED, "grouped_mm: built with %d registers per thread", a.numRegs);
  return GQ_OK;
}

template <int kForm>
gq_status setup_form() {
  gq_status st = setup_kernel<kForm, 1, false>();
  if (st == GQ_OK) st = setup_kernel<kForm, 2, false>();
  if constexpr (may_split(kForm))
    if (st == GQ_OK) st = setup_kernel<kForm, 1, true>();
  return st;
}

}  // namespace

gq_status setup(DeviceInfo& info) {
  for (const gq_status st : {setup_form<kForward>(), setup_form<kTransposed>(), setup_form<kGated>(),
                             setup_form<kGatedGrad>()})
    if (st != GQ_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(info.sm_count / 2 * 2));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<2>();
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const gq_status st = check_cuda(
      cudaOccupancyMaxActiveClusters(&info.mm_pairs, product_kernel<kForward, 2, false>, &cfg),
      "grouped_mm: resident block pairs");
  if (st != GQ_OK) return st;
  if (info.mm_pairs < 1) info.mm_pairs = 1;
  return setup_few(info);
}

namespace {

// Parameters of a product of rows of `inner` columns with E matrices (N, K), or
// pairs of them.
Params params_of(const DeviceInfo& info, const DebugKnobs& dbg, int form, const float* sa,
                 int64_t M, const float* sb, int32_t N, int32_t K, const int32_t* offs, int32_t E,
                 void* out) {
  const int32_t nb_n = (N + kBlock - 1) / kBlock, nb_k = (K + kBlock - 1) / kBlock;
  const bool transposed = is_transposed(form);
  Params p = {};
  p.form = form;
  p.inner = transposed ? N : K;
  p.outer = transposed ? K : N;
  p.sa = sa;
  p.sb = sb;
  p.offs = offs;
  p.out = static_cast<uint16_t*>(out);
  p.err = info.err_word;
  p.M = static_cast<int32_t>(M);
  p.E = E;
  p.kb_half = transposed ? nb_n : nb_k;
  p.kbs = form == kGatedGrad ? 2 * p.kb_half : p.kb_half;
  // the blocks of a pair of matrices follow each other along N, so that both
  // halves of a contraction over N are one run of blocks
  p.sb_expert = static_cast<int64_t>(nb_n) * nb_k * (form == kGatedGrad ? 2 : 1);
  p.sb_c = transposed ? 1 : nb_k;
  p.sb_k = transposed ? nb_k : 1;
  p.sb_last = (transposed ? nb_k : nb_n) - 1;
  p.sa_vec = p.kbs % kScaleKb == 0 && (reinterpret_cast<uintptr_t>(sa) & 15) == 0;
  p.timeout_ns = dbg.timeout_ns;
  p.skip_arrival = dbg.skip_arrival;
  return p;
}

template <int kForm, int kBlocks>
gq_status launch_many(const DeviceInfo& info, Params& p, const void* qa, const void* qb, int32_t N,
                      int32_t K, cudaStream_t stream) {
  constexpr int kTileCols = kForm == kGated ? kCols / 2 : kCols;
  p.tiles_c = (p.outer + kTileCols - 1) / kTileCols;
  const int64_t filled = p.E < p.M ? p.E : p.M;  // groups that have rows, at most
  const int64_t most = (p.M + filled * (kBlocks * kRows - 1)) / (kBlocks * kRows) * p.tiles_c;
  if (most > INT32_MAX)  // tiles of any offsets
    return fail(GQ_ERR_UNSUPPORTED, "grouped_mm: %lld tiles", static_cast<long long>(most));
  CUtensorMap amap, amap32, wmap;
  gq_status st = GQ_OK;
  for (CUtensorMap* m : {&amap, &amap32}) {
    st = encode_rows(m, p, qa, m == &amap ? kRows : kBoxRows);
    if (st != GQ_OK) return st;
  }
  st = encode_weights(&wmap, p, qb, N, K);
  if (st != GQ_OK) return st;
  if constexpr (kBlocks == 1 && may_split(kForm)) {
    const int32_t parts = p.kbs > kSplitKbs ? parts_of(info, p, most, kMostParts) : 1;
    if (parts > 1)
      return launch_chained("grouped_mm: launch", product_kernel<kForm, 1, true>,
                            dim3(static_cast<unsigned>(most * parts)), kThreads, smem_bytes<1>(),
                            stream, parts, amap, amap32, wmap, p);
  }
  const int resident = kBlocks == 2 ? info.mm_pairs : info.sm_count;
  const unsigned grid = kBlocks * static_cast<unsigned>(most < resident ? most : resident);
  return launch_chained("grouped_mm: launch", product_kernel<kForm, kBlocks, false>, dim3(grid), kThreads,
                        smem_bytes<kBlocks>(), stream, kBlocks, amap, amap32, wmap, p);
}

template <int kForm>
gq_status launch_form(const DeviceInfo& info, Params& p, const void* qa, const void* qb, int32_t N,
                      int32_t K, cudaStream_t stream) {
  constexpr int kFew = kForm == kGated ? kFewRowsGated : kFewRows;
  if (p.M <= static_cast<int64_t>(kFew) * p.E) return launch_few(info, p, qa, qb, N, K, stream);
  constexpr int kTileCols = kForm == kGated ? kCols / 2 : kCols;
  const int64_t tiles = static_cast<int64_t>(p.M) / kRows * ((p.outer + kTileCols - 1) / kTileCols);
  if ((p.inner % 64 != 0 || K % 64 != 0) && p.M > static_cast<int64_t>(kPairRows) * p.E &&
      tiles > static_cast<int64_t>(kPairTiles) * info.sm_count) {
    p.pairs_over = kPairRows * p.E;
    p.pairs_only = 1;
    const gq_status st = launch_many<kForm, 2>(info, p, qa, qb, N, K, stream);
    if (st != GQ_OK || !may_choose(kForm)) return st;
    p.pairs_only = -1;
  }
  return launch_many<kForm, 1>(info, p, qa, qb, N, K, stream);
}

}  // namespace

// Rows of the A operand: two dimensions, or for kGatedGrad three, so that a box
// that ends behind the last column of one half reads zeros, not the other half.
gq_status encode_rows(CUtensorMap* map, const Params& p, const void* qa, uint32_t rows) {
  const uint64_t inner = static_cast<uint64_t>(p.inner), m = static_cast<uint64_t>(p.M);
  if (p.form == kGatedGrad)
    return encode_tiled_3d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<void*>(qa), inner, 2, m,
                           inner, 2 * inner, kBlock, 1, CU_TENSOR_MAP_SWIZZLE_128B, rows);
  return encode_tiled_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<void*>(qa), inner, m, inner,
                         kBlock, rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Three dimensions: rows and columns past a matrix's own read zeros, never the
// next matrix's (a NaN there would survive the product with zero).
gq_status encode_weights(CUtensorMap* map, const Params& p, const void* qb, int32_t N, int32_t K) {
  const uint64_t count = static_cast<uint64_t>(p.E) * (p.form >= kGated ? 2 : 1);
  return encode_tiled_3d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<void*>(qb),
                         static_cast<uint64_t>(K), static_cast<uint64_t>(N), count,
                         static_cast<uint64_t>(K), static_cast<uint64_t>(N) * K, kBlock, kBlock,
                         CU_TENSOR_MAP_SWIZZLE_128B);
}

gq_status launch(const DeviceInfo& info, const DebugKnobs& dbg, const void* qa, const float* sa,
                 int64_t M, const void* qb, const float* sb, int32_t N, int32_t K, bool transposed,
                 const int32_t* offs, int32_t E, void* out, cudaStream_t stream) {
  Params p = params_of(info, dbg, transposed ? kTransposed : kForward, sa, M, sb, N, K, offs, E, out);
  return transposed ? launch_form<kTransposed>(info, p, qa, qb, N, K, stream)
                    : launch_form<kForward>(info, p, qa, qb, N, K, stream);
}

gq_status launch_gated(const DeviceInfo& info, const DebugKnobs& dbg, const void* qa,
                       const float* sa, int64_t M, const void* qb, const float* sb, int32_t N,
                       int32_t K, int activation, const int32_t* offs, int32_t E, void* out,
                       void* q, float* scales, void* pre, bool pow2, cudaStream_t stream) {
  Params p = params_of(info, dbg, kGated, sa, M, sb, N, K, offs, E, out);
  p.q = static_cast<uint8_t*>(q);
  p.scales = scales;
  p.pre = static_cast<uint16_t*>(pre);
  p.act = gated::act_of(activation);
  p.pow2 = pow2;
  return launch_form<kGated>(info, p, qa, qb, N, K, stream);
}

gq_status launch_gated_grad(const DeviceInfo& info, const DebugKnobs& dbg, const void* qd,
                            const float* sd, int64_t M, const void* qb, const float* sb, int32_t N,
                            int32_t K, const int32_t* offs, int32_t E, void* out,
                            cudaStream_t stream) {
  Params p = params_of(info, dbg, kGatedGrad, sd, M, sb, N, K, offs, E, out);
  return launch_form<kGatedGrad>(info, p, qd, qb, N, K, stream);
}

}  // namespace gmm
}  // namespace gq
