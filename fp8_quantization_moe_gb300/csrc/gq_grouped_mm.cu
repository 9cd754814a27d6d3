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
// The product is formed transposed: the weights are the MMA's M operand
// (256 output columns, 128 per block of the pair) and the rows (tokens) its
// N operand, so that a tile takes 16 to 160 tokens in steps of 16 and a
// group of any size wastes less than 16 rows.  A group of g tokens is cut
// into ceil(g / 160) tiles of equal size (to 16 tokens).
//
// Two blocks of a cluster share a tile (cta_group::2): each loads its 128
// weight rows and half of the tokens, 128 contraction columns at a time, and
// the pair's MMAs read both halves: per block and 128-column step 32 KB
// cross the shared memory instead of the 48 KB that one block alone needs
// for a tile of the same shape per SM, which would bind (128 bytes a cycle).
//
// Warp roles, per block:
//   0-15  epilogue: lane quarter w % 4 (32 output columns), token quarter
//         w / 4;
//   16    TMA loads (one lane);
//   17    TMEM allocation; in the pair's first block the MMAs (one lane);
//   18-19 the factors 1/sa * 1/sb of a tile, four 128-blocks at a time, into
//         a ring in shared memory.
// Every mbarrier wait is bounded; on expiry the error word is set, the warp
// leaves its loop and the others time out in turn.
#include <cuda_bf16.h>

#include "gq_device.cuh"
#include "gq_internal.h"
#include "gq_tcgen05.cuh"

namespace gq {
namespace gmm {

constexpr int kBlock = 128;       // contraction columns per scale, and per stage
constexpr int kRowsW = 128;       // output columns per block of a pair
constexpr int kUnit = 16;         // tokens per step of a tile's size
constexpr int kMaxN = 160;        // tokens of a tile
constexpr int kBufs = 512 / kMaxN;  // accumulators in TMEM
constexpr int kBoxLong = kMaxN / 2;  // tokens per TMA box: a block's half of a tile,
constexpr int kBoxShort = 16;     // or several of these
constexpr int kSubK = 32;         // contraction columns per MMA (kind::f8f6f4)
constexpr int kStages = 7;
constexpr int kWBytes = kRowsW * kBlock;           // 16 KB
constexpr int kTokBytes = kMaxN / 2 * kBlock;      // 10 KB
constexpr int kStageBytes = kWBytes + kTokBytes;
constexpr uint32_t kTmemCols = 512;
constexpr int kEpiWarps = 8;      // two per TMEM lane quarter
constexpr int kWarpUnits = kMaxN / kUnit / 2;
constexpr int kThreads = (kEpiWarps + 4) * 32;
constexpr int kScaleKb = 4;       // 128-blocks per entry of the factor ring
constexpr int kScaleRing = 2;
static_assert(kBufs * kMaxN <= 512 && kStageBytes % 1024 == 0, "TMEM columns, swizzle atoms");

struct Smem {
  uint8_t stage[kStages][kStageBytes];  // 1024-byte aligned (swizzle atoms)
  alignas(16) float factor[kScaleRing][kScaleKb][kMaxN];
  alignas(16) uint8_t rows[kEpiWarps][kUnit * 64];
  int32_t ends[kMaxGroups];
  int32_t first[kMaxGroups + 1];  // token tiles before each group
  uint64_t full[kStages];         // both blocks' loads (the pair's first block)
  uint64_t done[kStages];         // the stage's MMAs are complete (commit, both blocks):
                                  // the stage is free, its accumulator full
  uint64_t acc_empty[kBufs];        // accumulator read (16 warps; the first block)
  uint64_t fac_full[kScaleRing];
  uint64_t fac_empty[kScaleRing];
  uint64_t drain;
  uint32_t tmem_base;
};
constexpr size_t kSmemBytes = sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "fits one SM's shared memory");

struct Params {
  const float* sa;
  const float* sb;
  const int32_t* offs;
  uint16_t* out;
  unsigned* err;
  int32_t M, E, inner, outer;
  int32_t kbs;                 // 128-blocks of the contraction
  int32_t tiles_c;             // 256-column tiles of the output
  int64_t sb_expert;           // scales per expert
  int32_t sb_c, sb_k;          // scale strides along output and contraction blocks
  int32_t sb_last;             // last output block
  bool sa_vec;                 // rows of sa are 16-byte aligned
  bool transposed;
  uint64_t timeout_ns;
  int32_t skip_arrival;        // test hook: block 0 never frees its first accumulator
};

struct Tile {
  int32_t g, c0, t0, tokens, n;  // group, first column, first token, its tokens, the MMA's N
};

__device__ __forceinline__ Tile tile_of(const Params& p, const Smem& s, int64_t i) {
  // the last group whose first tile is at or before i
  int32_t lo = 0, hi = p.E;
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (static_cast<int64_t>(s.first[mid]) * p.tiles_c <= i) lo = mid; else hi = mid;
  }
  Tile t;
  t.g = lo;
  const int32_t tt = s.first[lo + 1] - s.first[lo];
  const int32_t r = static_cast<int32_t>(i - static_cast<int64_t>(s.first[lo]) * p.tiles_c);
  const int32_t start = lo > 0 ? s.ends[lo - 1] : 0;
  const int32_t size = s.ends[lo] - start;
  const int64_t units = (size + kUnit - 1) / kUnit;
  const int32_t j = r % tt;
  const int32_t u0 = static_cast<int32_t>(units * j / tt);
  const int32_t u1 = static_cast<int32_t>(units * (j + 1) / tt);
  t.c0 = (r / tt) * 2 * kRowsW;
  t.t0 = start + u0 * kUnit;
  t.n = (u1 - u0) * kUnit;
  t.tokens = min(t.n, size - u0 * kUnit);
  return t;
}

// Where token j's factor lies: the order in which a lane of the 16x128b TMEM
// layout needs them, so that one 16-byte load gives its four of 16 tokens.
__device__ __forceinline__ int factor_slot(int j) {
  return (j & ~15) | ((j & 3) << 2) | ((j >> 2) & 3);
}

constexpr uint32_t kIdescBase = (1u << 4) | (16u << 24);  // D fp32, e4m3 x e4m3, M = 256

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap amap,
                   const __grid_constant__ CUtensorMap amap16,
                   const __grid_constant__ CUtensorMap wmap, const Params p) {
  // aligned by an offset, so that the compiler still knows the address space
  extern __shared__ uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>(smem_raw + (-smem_addr(smem_raw) & 1023u));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const uint64_t wait_ns = 4 * p.timeout_ns;

  if (warp == kEpiWarps) {
    build_ends(p.offs, 0, p.E, p.M, s.ends, lane);
    __syncwarp();
    int32_t carry = 0;
    for (int base = 0; base < p.E; base += 32) {
      const int g = base + lane;
      int32_t v = 0;
      if (g < p.E) v = (s.ends[g] - (g > 0 ? s.ends[g - 1] : 0) + kMaxN - 1) / kMaxN;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int32_t o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += o;
      }
      if (g < p.E) s.first[g + 1] = carry + v;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) {
      s.first[0] = 0;
      prefetch_tensormap(&amap);
      prefetch_tensormap(&amap16);
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
      mbar_init(&s.fac_full[i], 2);
      mbar_init(&s.fac_empty[i], kEpiWarps);
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
  const int64_t tiles = static_cast<int64_t>(s.first[p.E]) * p.tiles_c;
  const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (warp >= kEpiWarps) {
    setmaxnreg_dec<72>();
    if (warp == kEpiWarps) {
      // ---------------------------------------------------------- loads --
      const uint64_t pol = policy_evict_normal();
      const uint32_t done = smem_addr(s.done), full = map_cluster(smem_addr(s.full), 0);
      uint32_t st = 0, use = 0;  // stage, its use
      bool ok = true;
      for (int64_t i = pair; ok && i < tiles; i += pairs) {
        const Tile t = tile_of(p, s, i);
        const int32_t half = t.n / 2;
        // one long box reads up to half of its rows for nothing
        const int boxes = half > kBoxLong / 2 ? 0 : (half + kBoxShort - 1) / kBoxShort;
        const uint32_t bytes =
            2u * (kWBytes + (boxes == 0 ? kBoxLong : boxes * kBoxShort) * kBlock);
        const int32_t tok = t.t0 + static_cast<int32_t>(rank) * half;
        const int32_t c = t.c0 + static_cast<int32_t>(rank) * kRowsW;
        for (int32_t k = 0; k < p.inner; k += kBlock) {
          ok = mbar_wait_warp(done + st * 8, (use & 1) ^ 1u, wait_ns, p.err);
          if (!ok) break;
          if (elect_one()) {
            uint8_t* base = s.stage[st];
            if (rank == 0)  // both blocks' bytes complete on the first block's barrier
              mbar_arrive_expect_tx(&s.full[st], bytes);
            const uint32_t bar = full + st * 8;
            tma_load_3d_pair(base, &wmap, p.transposed ? c : k, p.transposed ? k : c, t.g, bar, pol);
            if (boxes == 0)
              tma_load_2d_pair(base + kWBytes, &amap, k, tok, bar, pol);
            for (int b = 0; b < boxes; ++b)
              tma_load_2d_pair(base + kWBytes + b * kBoxShort * kBlock, &amap16, k,
                               tok + b * kBoxShort, bar, pol);
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
        for (int64_t i = pair; ok && i < tiles; i += pairs) {
          const Tile t = tile_of(p, s, i);
          const uint32_t n = __shfl_sync(0xffffffffu, static_cast<uint32_t>(t.n), 0);
          const uint32_t idesc = kIdescBase | ((n >> 3) << 17) | (p.transposed ? 1u << 15 : 0u);
          for (int32_t left = p.inner; left > 0; left -= kBlock) {
            ok = mbar_wait_warp(acc_empty + b * 8, (use & 1) ^ 1u, wait_ns, p.err) &&
                 mbar_wait_warp(full + st * 8, st_use & 1, wait_ns, p.err);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              const uint32_t d = tmem + b * kMaxN;
              // weights: K-major rows of 128 bytes, or MN-major (32
              // contraction rows = 4 KB); tokens: K-major
              const uint32_t w0 = stage0 + st * kStageBytes;
              uint64_t wd = operand_desc_sw128(w0, 1024u);
              uint64_t ad = operand_desc_sw128(w0 + kWBytes, 1024u);
              tc_mma_e4m3_pair<false>(d, wd, ad, idesc);
#pragma unroll
              for (int j = 1; j < kBlock / kSubK; ++j) {
                wd += wstep;
                ad += kSubK >> 4;
                if (j * kSubK < left) tc_mma_e4m3_pair<true>(d, wd, ad, idesc);
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
    } else {
      // -------------------------------------------------------- factors --
      // Two warps, every other 32 tokens each; the scales of an entry (a
      // tile's next four 128-blocks) are loaded while the one before is
      // worked on.
      constexpr int kQ = (kMaxN + 63) / 64;  // tokens per lane
      const int32_t first = (warp - kEpiWarps - 2) * 32 + lane;
      float v[kQ][kScaleKb], rb[kScaleKb];
      int64_t i = pair;
      int32_t kb = 0, n = 0;
      Tile t = {};
      auto load = [&]() {  // the entry (tile i, 128-blocks kb ..)
        if (kb == 0) t = tile_of(p, s, i);
        const int32_t cb = min(t.c0 / kBlock + static_cast<int32_t>(rank), p.sb_last);
        const float* sb = p.sb + t.g * p.sb_expert + static_cast<int64_t>(cb) * p.sb_c;
#pragma unroll
        for (int u = 0; u < kScaleKb; ++u)
          rb[u] = __ldg(sb + static_cast<int64_t>(min(kb + u, p.kbs - 1)) * p.sb_k);
#pragma unroll
        for (int q = 0; q < kQ; ++q) {
          const int32_t row = min(t.t0 + min(first + 64 * q, t.n - 1), p.M - 1);
          const float* src = p.sa + static_cast<int64_t>(row) * p.kbs;
          if (p.sa_vec) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(src + kb));
            v[q][0] = x.x;
            v[q][1] = x.y;
            v[q][2] = x.z;
            v[q][3] = x.w;
          } else {
#pragma unroll
            for (int u = 0; u < kScaleKb; ++u) v[q][u] = __ldg(src + min(kb + u, p.kbs - 1));
          }
        }
        n = t.n;
      };
      uint32_t e = 0;
      bool ok = true;
      if (i < tiles) load();
      while (i < tiles) {
        const int r = static_cast<int>(e % kScaleRing);
        float f[kQ][kScaleKb];
#pragma unroll
        for (int u = 0; u < kScaleKb; ++u) {
          const float w = rcp_approx(rb[u]);
#pragma unroll
          for (int q = 0; q < kQ; ++q) f[q][u] = __fmul_rn(rcp_approx(v[q][u]), w);
        }
        const int32_t have = n;
        kb += kScaleKb;
        if (kb >= p.kbs) {
          kb = 0;
          i += pairs;
        }
        if (i < tiles) load();
        ok = __all_sync(0xffffffffu, mbar_wait(&s.fac_empty[r], ((e / kScaleRing) & 1) ^ 1u,
                                               wait_ns, p.err));
        if (!ok) break;
#pragma unroll
        for (int q = 0; q < kQ; ++q) {
          const int32_t j = first + 64 * q;
          if (j < have) {
#pragma unroll
            for (int u = 0; u < kScaleKb; ++u) s.factor[r][u][factor_slot(j)] = f[q][u];
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.fac_full[r]);
        ++e;
      }
    }
  } else {
    // --------------------------------------------------------- epilogue --
    // The 16x128b TMEM layout: of 16 lanes (output columns) and 4 tokens,
    // lane l of the warp holds token l % 4 of output columns l / 4 and
    // l / 4 + 8.  acc[u][g][r]: token 16 u + 4 g + l % 4 of this warp's,
    // output column l / 4 + 8 r of its lane quarter.
    //
    // A 128-block's values are all loaded into registers, the accumulator is
    // given back to the MMAs, and only then scaled and added.
    setmaxnreg_inc<216>();
    const int q = warp & 3, part = warp >> 2;
    const uint32_t lane_base = static_cast<uint32_t>(32 * q) << 16;
    const uint32_t stage_rows = smem_addr(s.rows[warp]);
    const uint32_t done = smem_addr(s.done), fac_full = smem_addr(s.fac_full);
    const uint32_t acc_empty = map_cluster(smem_addr(s.acc_empty), 0);
    const uint32_t factors = smem_addr(s.factor) + (lane & 3) * 16;
    uint32_t b = 0;             // accumulator
    uint32_t st = 0, use = 0;   // the stage whose MMAs filled it, its use
    uint32_t e = 0;           // entries of the factor ring so far
    bool first = p.skip_arrival && blockIdx.x == 0;  // withhold the next release
    bool ok = true;
    for (int64_t i = pair; ok && i < tiles; i += pairs) {
      const Tile t = tile_of(p, s, i);
      const int32_t units = t.n / kUnit, half = (units + 1) / 2;
      const int32_t j0 = part * half * kUnit;                // this warp's first token
      const int32_t mine = part == 0 ? half : units - half;  // and its units
      const uint32_t tacc0 = tmem + lane_base + static_cast<uint32_t>(j0);
      float acc[kWarpUnits][4][4];
#pragma unroll
      for (int a = 0; a < 16 * kWarpUnits; ++a) acc[a / 16][a / 4 % 4][a % 4] = 0.0f;
      int32_t left = p.kbs;
      while (left > 0) {
        const uint32_t r = e % kScaleRing;
        if (!mbar_wait_warp(fac_full + r * 8, (e / kScaleRing) & 1, wait_ns, p.err)) break;
        const int32_t kbs = min(left, kScaleKb);
        uint32_t fac = factors + (r * kScaleKb * kMaxN + j0) * 4;
        int32_t v = 0;
        for (; v < kbs; ++v, fac += kMaxN * 4) {
          if (!mbar_wait_warp(done + st * 8, use & 1, wait_ns, p.err)) break;
          tc_fence_after();
          const uint32_t tacc = tacc0 + b * kMaxN;
          uint32_t lo[kWarpUnits][8], hi[kWarpUnits][8];
          uint4 f[kWarpUnits];
#pragma unroll
          for (int u = 0; u < kWarpUnits; ++u) {
            tmem_ld_16x128b_x4(tacc + u * kUnit, lo[u]);
            tmem_ld_16x128b_x4(tacc + (16u << 16) + u * kUnit, hi[u]);
          }
#pragma unroll
          for (int u = 0; u < kWarpUnits; ++u) f[u] = lds128_ordered(fac + u * kUnit * 4);
          tmem_ld_wait();
#pragma unroll
          for (int u = 0; u < kWarpUnits; ++u) {
            pin8(lo[u]);
            pin8(hi[u]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0 && !first) mbar_arrive_cluster(acc_empty + b * 8);
          first = false;
          if (++b == kBufs) b = 0;
          if (++st == kStages) {
            st = 0;
            ++use;
          }
#pragma unroll
          for (int u = 0; u < kWarpUnits; ++u) {
              const float w[4] = {__uint_as_float(f[u].x), __uint_as_float(f[u].y),
                                  __uint_as_float(f[u].z), __uint_as_float(f[u].w)};
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                acc[u][g][0] = __fmaf_rn(__uint_as_float(lo[u][2 * g]), w[g], acc[u][g][0]);
                acc[u][g][1] = __fmaf_rn(__uint_as_float(lo[u][2 * g + 1]), w[g], acc[u][g][1]);
                acc[u][g][2] = __fmaf_rn(__uint_as_float(hi[u][2 * g]), w[g], acc[u][g][2]);
                acc[u][g][3] = __fmaf_rn(__uint_as_float(hi[u][2 * g + 1]), w[g], acc[u][g][3]);
              }
            }
        }
        if (v < kbs) break;
        if (lane == 0) mbar_arrive(&s.fac_empty[r]);
        ++e;
        left -= kbs;
      }
      ok = left <= 0;
      if (!ok) break;
      // 16 tokens at a time: transposed into token rows of 64 bytes (32
      // output columns) in the staging buffer, whose 16-byte parts are
      // XOR-swizzled by (token / 2) % 4, then stored eight rows per step
      const int32_t c = t.c0 + static_cast<int32_t>(rank) * kRowsW + 32 * q;
      const int col = lane & 3;
      const bool c_ok = c + col * 8 < p.outer;  // outer % 16 == 0: whole parts
#pragma unroll
      for (int u = 0; u < kWarpUnits; ++u) {
        if (u >= mine) continue;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint32_t w[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) w[r] = bf16x2_of(acc[u][2 * g][r], acc[u][2 * g + 1][r]);
          const int tok = 8 * g + 4 * (lane & 1) + ((lane & 7) >> 1);
          stmatrix_x4_trans(stage_rows + tok * 64 + (((lane >> 3) ^ ((tok >> 1) & 3)) << 4), w);
        }
        __syncwarp();
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int tok = 8 * g + (lane >> 2);
          const uint4 v = lds128_ordered(stage_rows + tok * 64 + ((col ^ ((tok >> 1) & 3)) << 4));
          const int32_t j = j0 + u * kUnit + tok;
          if (j < t.tokens && c_ok)
            *reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(t.t0 + j) * p.outer + c +
                                      col * 8) = v;
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
  return GQ_OK;
}

gq_status launch(const DeviceInfo& info, const DebugKnobs& dbg, const void* qa, const float* sa,
                 int64_t M, const void* qb, const float* sb, int32_t N, int32_t K, bool transposed,
                 const int32_t* offs, int32_t E, void* out, cudaStream_t stream) {
  Params p;
  p.inner = transposed ? N : K;
  p.outer = transposed ? K : N;
  CUtensorMap amap, amap16, wmap;
  gq_status st = GQ_OK;
  for (CUtensorMap* m : {&amap, &amap16}) {
    st = encode_tiled_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<void*>(qa),
                         static_cast<uint64_t>(p.inner), static_cast<uint64_t>(M),
                         static_cast<uint64_t>(p.inner), kBlock, m == &amap ? kBoxLong : kBoxShort,
                         CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != GQ_OK) return st;
  }
  // three dimensions: rows and columns past an expert's own read zeros, never
  // the next expert's (a NaN there would survive the product with zero)
  st = encode_tiled_3d(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<void*>(qb),
                       static_cast<uint64_t>(K), static_cast<uint64_t>(N), static_cast<uint64_t>(E),
                       static_cast<uint64_t>(K), static_cast<uint64_t>(N) * K, kBlock, kRowsW,
                       CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != GQ_OK) return st;
  const int32_t nb_n = (N + kBlock - 1) / kBlock, nb_k = (K + kBlock - 1) / kBlock;
  p.sa = sa;
  p.sb = sb;
  p.offs = offs;
  p.out = static_cast<uint16_t*>(out);
  p.err = info.err_word;
  p.M = static_cast<int32_t>(M);
  p.E = E;
  p.kbs = (p.inner + kBlock - 1) / kBlock;
  p.tiles_c = (p.outer + 2 * kRowsW - 1) / (2 * kRowsW);
  p.sb_expert = static_cast<int64_t>(nb_n) * nb_k;
  p.sb_c = transposed ? 1 : nb_k;
  p.sb_k = transposed ? nb_k : 1;
  p.sb_last = (transposed ? nb_k : nb_n) - 1;
  p.sa_vec = p.kbs % kScaleKb == 0 && (reinterpret_cast<uintptr_t>(sa) & 15) == 0;
  p.transposed = transposed;
  p.timeout_ns = dbg.timeout_ns;
  p.skip_arrival = dbg.skip_arrival;
  const int64_t most = (M / kMaxN + (E < M ? E : M)) * p.tiles_c;  // tiles of any offsets
  const int64_t pairs = most < info.mm_pairs ? most : info.mm_pairs;
  product_kernel<<<static_cast<unsigned>(2 * pairs), kThreads, kSmemBytes, stream>>>(amap, amap16, wmap,
                                                                                       p);
  return check_cuda(cudaGetLastError(), "grouped_mm: launch");
}

}  // namespace gmm
}  // namespace gq
