// gq_grouped_mm_few.cu -- the grouped block-scaled product where the groups
// have few rows (decoding): every touched expert's weights are read once for
// a handful of rows, so HBM bounds it, 1 byte per weight.  512 rows of 64
// experts, K 2064 to N 2832: 59 us, 6.4 TB/s; eight rows of eight experts, K
// 2048 to N 4096: 14.3 us, of which 9.9 us are the weights and most of the
// rest the launch, the first loads and the last tile.
//
// In the gated form a tile has 128 columns of both projections and up to 64 rows:
// one token to eight of 64 experts, 2 x 2048 x 4096, 134 MB: 24.3 us, of which the
// loads take 21.4; 512 rows of 64 experts, 2 x 1424 x 2064: 58.3 us, 6.5 TB/s (fp8
// 60).
//
// Here the weights are the MMA's M operand (128 output columns) and the rows
// its N operand, up to 128 of them in steps of 16: an MMA costs as many cycles
// as there are rows, and four accumulators keep the tensor cores, the epilogue
// and 96 KB of weights per SM in flight at once.  A lane of the epilogue owns
// an output column and needs every row's factor 1/sa * 1/sb; with few rows
// those shared loads are cheap.
//
// One persistent block per SM -- or, where the gated forms have few tiles, a cluster
// per tile (see Split) -- whose warps are:
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
constexpr int kUnit = 16;      // rows of a tile come in units
constexpr int kWBytes = kCols * kBlock;   // 16 KB
constexpr int kScaleRing = 4;
constexpr int kMostParts = 8;  // blocks that share a tile, at most
constexpr int kEpiWarps = 8;
constexpr int kThreads = (kEpiWarps + 3) * 32;

// kGated: a tile has the columns of both projections, two MMAs with the same
// rows; half as many of these, so that TMEM holds four accumulators all the same.
template <int kForm>
struct Sizes {
  static constexpr int kMats = kForm == kGated ? 2 : 1;
  static constexpr int kTok = 128 / kMats;       // rows of a tile, at most (the MMA's N)
  static constexpr int kWarpTok = kTok / 2;      // rows of an epilogue warp, at most
  static constexpr int kStageBytes = kMats * kWBytes + kTok * kBlock;
  static constexpr int kStages = kForm == kGated ? 5 : 6;
  static constexpr int kAccCols = kMats * kTok;  // TMEM columns of an accumulator
  static constexpr int kBufs = 512 / kAccCols;
  static_assert(kEpiWarps == 4 * (kTok / kWarpTok), "two warps per lane quarter");
};
// Accumulators in use: of a split tile three, so that also a block with one entry of
// four 128-blocks waits for a release, and notices one that does not come.
template <int kForm, bool kSplit>
constexpr uint32_t kBufsOf = kSplit ? 3 : Sizes<kForm>::kBufs;

template <int kForm>
struct Smem {
  using Z = Sizes<kForm>;
  static constexpr int kStages = Z::kStages, kBufs = Z::kBufs;
  uint8_t stage[kStages][Z::kStageBytes];
  alignas(16) float factor[kScaleRing][kScaleKb][Z::kAccCols];  // kGated: of both matrices
  TileTable tiles;
  uint64_t full[kStages];
  uint64_t done[kStages];
  uint64_t acc_empty[kBufs];
  uint64_t fac_full[kScaleRing];
  uint64_t fac_empty[kScaleRing];
  uint64_t drain;
  uint64_t pair[2];              // kGated: the four warps of a row have their maxima
  alignas(16) float most[2][2][Z::kWarpTok][4];  // kGated: those, by exchange parity, warps' rows
  uint32_t tmem_base;
};
template <int kForm>
constexpr size_t smem_bytes() {
  static_assert(sizeof(Smem<kForm>) + 1024 <= 227 * 1024, "fits one SM's shared memory");
  return sizeof(Smem<kForm>) + 1024;
}

template <int kForm>
__device__ __forceinline__ int32_t units_of(const Tile& t) {
  return (min(t.rows, Sizes<kForm>::kTok) + kUnit - 1) / kUnit;
}

// Positions in the rings, common to a tile's steps.
struct Rings {
  uint32_t b = 0;              // accumulator
  uint32_t st = 0, use = 0;    // stage, its use
  uint32_t r = 0, sc_use = 0;  // entry of the factor ring, its use
  uint32_t shares = 0;         // kGated: exchanges of maxima so far
  bool hold = false;           // test hook: withhold the next release
  bool joined = false;         // split: this warp has met the cluster's barrier
};

// Rows of 128-columns' values in TMEM lanes (a lane is a column c) to bf16 rows:
// four rows at a time; two exchanges among four neighbouring lanes leave each with
// four columns of one of the rows, so that a store covers 64 bytes of all four.
// `out` points at column (c & ~3) of row (lane & 3).
template <int kN>
__device__ __forceinline__ void store_bf16(const float (&v)[kN][kUnit], uint16_t* out, int64_t pitch,
                                           int32_t rows, bool c_ok, const Split& part, int lane) {
  const bool high = lane & 2, odd = lane & 1;
#pragma unroll
  for (int u = 0; u < kN; ++u)
#pragma unroll
    for (int j = 0; j < kUnit; j += 4) {
      if (u * kUnit + j >= rows || !part.mine((u * kUnit + j) / 4)) continue;  // rows may end early
      const uint32_t w0 = bf16x2_of(v[u][j], v[u][j + 1]), w1 = bf16x2_of(v[u][j + 2], v[u][j + 3]);
      // two of the rows, of columns c and c ^ 2, then one of columns c and c ^ 2, c ^ 1 and c ^ 3
      const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? w0 : w1, 2);
      const uint32_t lo = high ? got : w0, hi = high ? w1 : got;  // columns 0 or 1, and 2 or 3
      const uint32_t keep = __byte_perm(lo, hi, odd ? 0x7632 : 0x5410);
      const uint32_t back = __shfl_xor_sync(0xffffffffu, __byte_perm(lo, hi, odd ? 0x5410 : 0x7632), 1);
      const uint32_t even = odd ? back : keep, other = odd ? keep : back;  // columns 0 and 2, 1 and 3
      if (u * kUnit + j + (lane & 3) < rows && c_ok)
        *reinterpret_cast<uint2*>(out + static_cast<int64_t>(u * kUnit + j) * pitch) =
            make_uint2(__byte_perm(even, other, 0x5410), __byte_perm(even, other, 0x7632));
    }
}

// kGated: the rows of a tile, x and u (columns in lanes), to what is asked for.
template <int kN>
__device__ __forceinline__ bool gated_store(const Params& p, const Split& part, Smem<kGated>& s,
                                            const Tile& t, Rings& r,
                                            float (&x)[kN][kUnit], float (&u)[kN][kUnit], int32_t j0,
                                            int q, int lane, uint64_t wait_ns) {
  const int32_t rows = t.rows - j0;
  const int32_t c = t.c0 + 32 * q + lane, four = c & ~3, of_four = lane & 3;
  const bool c_ok = four < p.outer;  // outer % 16 == 0
  const int64_t row = t.m0 + j0, n = p.outer;
  if (p.pre != nullptr) {
    uint16_t* const to = p.pre + (row + of_four) * 2 * n + four;
    store_bf16(x, to, 2 * n, rows, c_ok, part, lane);
    store_bf16(u, to + n, 2 * n, rows, c_ok, part, lane);
  }
#pragma unroll
  for (int a = 0; a < kN; ++a) gated::gate(p.act, x[a], u[a]);
  if (p.out != nullptr) store_bf16(x, p.out + (row + of_four) * n + four, n, rows, c_ok, part, lane);
  if (p.q == nullptr) return true;
  // the maximum of a row over this warp's 32 columns, then over the four warps that
  // hold its 128 (a NaN does not count; columns past the last hold anything); with
  // five exchanges a row, and its scale formed by every lane, 1024 rows of 64
  // experts, 2 x 1024 x 2048, took 58 us, this way 48
  const int g = j0 / Sizes<kGated>::kWarpTok;
  float(*const most)[4] = s.most[r.shares & 1][g];
#pragma unroll
  for (int a = 0; a < kN; ++a) {
    uint32_t m = 0;  // of row `lane & 15`, bits: of values that are not negative in their order
#pragma unroll
    for (int j = 0; j < kUnit; j += 4) {
      if (a * kUnit + j >= rows || !part.mine((a * kUnit + j) / 4)) continue;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float v = c < p.outer ? fmaxf(fabsf(x[a][j + k]), 0.0f) : 0.0f;
        const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(v));
        if ((lane & 15) == j + k) m = top;
      }
    }
    if (lane < kUnit) sts32(smem_addr(&most[a * kUnit + lane][q]), __uint_as_float(m));
  }
  __syncwarp();
  if (lane == 0) mbar_arrive(&s.pair[g]);
  if (!mbar_wait_warp(smem_addr(&s.pair[g]), r.shares & 1, wait_ns, p.err)) return false;
  ++r.shares;
  const int32_t nb = (p.outer + kBlock - 1) / kBlock;
#pragma unroll
  for (int a = 0; a < kN; ++a) {
    if (a * kUnit >= rows) continue;
    // a row's scale is formed by one lane, which holds it for the others
    const int32_t own = lane & (kUnit - 1);
    const uint4 m = lds128_ordered(smem_addr(most[a * kUnit + own]));
    const float sc = scale_from_amax_bits(max(max(m.x, m.y), max(m.z, m.w)), p.pow2);
    if (q == 0 && lane < kUnit && a * kUnit + own < rows && part.mine((a * kUnit + own) / 4))
      p.scales[(row + a * kUnit + own) * nb + t.c0 / kBlock] = sc;
#pragma unroll
    for (int j = 0; j < kUnit; j += 4) {
      if (a * kUnit + j >= rows || !part.mine((a * kUnit + j) / 4)) continue;
      // four rows: a lane's bytes of its column, then by two exchanges of bytes the
      // bytes of four columns of one row, lane & 3
      uint32_t w = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float v = x[a][j + k];
        const float of = __shfl_sync(0xffffffffu, sc, j + k);
        w |= (quant4f(make_float4(v, v, v, v), of) & 0xFFu) << (8 * k);
      }
      uint32_t o = __shfl_xor_sync(0xffffffffu, w, 1);
      w = lane & 1 ? __byte_perm(w, o, 0x3715) : __byte_perm(w, o, 0x6240);
      o = __shfl_xor_sync(0xffffffffu, w, 2);
      w = lane & 2 ? __byte_perm(w, o, 0x3276) : __byte_perm(w, o, 0x5410);
      const int32_t at = a * kUnit + j + of_four;
      if (at < rows && c_ok) *reinterpret_cast<uint32_t*>(p.q + (row + at) * n + four) = w;
    }
  }
  return true;
}

// A tile of which this warp has kU * 16 rows from row j0 on (kU = 0: none, it
// only keeps step); false if a wait expired.
template <int kForm, bool kSplit, int kU>
__device__ __forceinline__ bool tile_body(const Params& p, const Split& part, Smem<kForm>& s,
                                          const Tile& t, Rings& x, uint32_t tmem0, int32_t j0,
                                          int q, int lane, uint64_t wait_ns) {
  using Z = Sizes<kForm>;
  constexpr int kN = kU > 0 ? kU : 1;
  float acc[Z::kMats][kN][kUnit];
#pragma unroll
  for (int i = 0; i < Z::kMats; ++i)
#pragma unroll
    for (int a = 0; a < kN * kUnit; ++a) acc[i][a / kUnit][a % kUnit] = 0.0f;
  const uint32_t done = smem_addr(s.done), fac_full = smem_addr(s.fac_full);
  const uint32_t factors = smem_addr(s.factor), acc_empty = smem_addr(s.acc_empty);
#pragma unroll 1
  for (int32_t kb = part.kb0; kb < part.kb1; ++kb) {
    const uint32_t e = kb % kScaleKb;
    if (e == 0 && !mbar_wait_warp(fac_full + x.r * 8, x.sc_use & 1, wait_ns, p.err)) return false;
    if (!mbar_wait_warp(done + x.st * 8, x.use & 1, wait_ns, p.err)) return false;
    tc_fence_after();
    uint32_t h[Z::kMats][kN][kUnit];
#pragma unroll
    for (int i = 0; i < Z::kMats; ++i)
#pragma unroll
      for (int u = 0; u < kU; ++u)
        tmem_ld_32x32b_x16(tmem0 + x.b * Z::kAccCols + i * Z::kTok + j0 + u * kUnit, h[i][u]);
#pragma unroll
    for (int i = 0; i < Z::kMats; ++i)
#pragma unroll
      for (int u = 0; u < kU; ++u) tmem_ld_wait16(h[i][u]);
    tc_fence_before();
    __syncwarp();
    if (lane == 0 && !x.hold) mbar_arrive_addr(acc_empty + x.b * 8);
    x.hold = false;
    const uint32_t fac = factors + ((x.r * kScaleKb + e) * Z::kAccCols + j0) * 4;
#pragma unroll
    for (int i = 0; i < Z::kMats; ++i)
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        uint4 f[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) f[v] = lds128_ordered(fac + (i * Z::kTok + u * kUnit + 4 * v) * 4);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float w[4] = {__uint_as_float(f[v].x), __uint_as_float(f[v].y),
                              __uint_as_float(f[v].z), __uint_as_float(f[v].w)};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[i][u][4 * v + j] =
                __fmaf_rn(__uint_as_float(h[i][u][4 * v + j]), w[j], acc[i][u][4 * v + j]);
        }
      }
    if (++x.b == kBufsOf<kForm, kSplit>) x.b = 0;
    if (++x.st == Z::kStages) {
      x.st = 0;
      ++x.use;
    }
    if (e == kScaleKb - 1 || kb == part.kb1 - 1) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.fac_empty[x.r]);
      if (++x.r == kScaleRing) {
        x.r = 0;
        ++x.sc_use;
      }
    }
  }
  if constexpr (kSplit) {
    // The stages are free: all MMAs of the block are complete.  Four rows of a
    // column are one 16-byte word.
    const uint32_t own = smem_addr(s.stage) + (j0 / 4 * kCols + 32 * q + lane) * 16;
    constexpr uint32_t kQuad = kCols * 16, kMat = Z::kTok / 4 * kQuad;
#pragma unroll
    for (int a = 0; a < kU * kUnit; a += 4)
      if (j0 + a < t.rows && !part.mine(a / 4))
#pragma unroll
        for (int i = 0; i < Z::kMats; ++i) {
          const float* v = &acc[i][a / kUnit][a % kUnit];
          sts128(own + i * kMat + a / 4 * kQuad,
                 make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                            __float_as_uint(v[3])));
        }
    cluster_arrive();
    cluster_wait();
    x.joined = true;
    uint32_t from[kMostParts];
#pragma unroll
    for (int r = 0; r < kMostParts; ++r) from[r] = map_cluster(own, min(r, part.parts - 1));
#pragma unroll
    for (int a = 0; a < kU * kUnit; a += 4) {
      if (j0 + a >= t.rows || !part.mine(a / 4)) continue;
#pragma unroll
      for (int i = 0; i < Z::kMats; ++i) {
        // of every block at once (of a missing one the last one's again), added in order
        uint4 v[kMostParts];
#pragma unroll
        for (int r = 0; r < kMostParts; ++r) v[r] = ld_cluster_128(from[r] + i * kMat + a / 4 * kQuad);
        float* const o = &acc[i][a / kUnit][a % kUnit];
        float sum[4] = {};
#pragma unroll
        for (int r = 0; r < kMostParts; ++r)
          if (r < part.parts) {
            const bool here = r == part.rank;  // in registers, not in shared memory
            sum[0] += here ? o[0] : __uint_as_float(v[r].x);
            sum[1] += here ? o[1] : __uint_as_float(v[r].y);
            sum[2] += here ? o[2] : __uint_as_float(v[r].z);
            sum[3] += here ? o[3] : __uint_as_float(v[r].w);
          }
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = sum[k];
      }
    }
  }
  if constexpr (kU == 0) {
    return true;
  } else if constexpr (kForm == kGated) {
    return gated_store<kU>(p, part, s, t, x, acc[0], acc[1], j0, q, lane, wait_ns);
  } else {
    const int32_t c = t.c0 + 32 * q + (lane & ~3);
    store_bf16<kU>(acc[0], p.out + static_cast<int64_t>(t.m0 + j0 + (lane & 3)) * p.outer + c, p.outer,
                   t.rows - j0, c < p.outer, part, lane);
    return true;
  }
}

template <int kForm, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    few_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap wmap,
               const Params p) {
  using Z = Sizes<kForm>;
  constexpr bool kT = is_transposed(kForm);
  constexpr int kTok = Z::kTok, kStages = Z::kStages;
  constexpr uint32_t kBufs = kBufsOf<kForm, kSplit>;
  extern __shared__ uint8_t smem_raw[];
  Smem<kForm>& s = *reinterpret_cast<Smem<kForm>*>(smem_raw + (-smem_addr(smem_raw) & 1023u));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  const Split part = split_of<kSplit>(p);
  const int32_t groups = gridDim.x / part.parts, group = blockIdx.x / part.parts;
  const uint64_t wait_ns = 4 * p.timeout_ns;

  if (warp == kEpiWarps && lane == 0) {
    prefetch_tensormap(&amap);
    prefetch_tensormap(&wmap);
  } else if (warp == kEpiWarps + 2 && lane == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.done[i], 1);
    }
    for (uint32_t b = 0; b < kBufs; ++b) mbar_init(&s.acc_empty[b], kEpiWarps);
    for (int i = 0; i < kScaleRing; ++i) {
      mbar_init(&s.fac_full[i], 1);
      mbar_init(&s.fac_empty[i], kEpiWarps);
    }
    mbar_init(&s.drain, 1);
    for (int i = 0; i < 2; ++i) mbar_init(&s.pair[i], 4);
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

  bool joined = false;
  if (warp == kEpiWarps) {
    // ------------------------------------------------------------ loads --
    const uint64_t pol_w = policy_evict_first(), pol_a = policy_evict_last();
    const uint32_t done = smem_addr(s.done);
    uint32_t st = 0, use = 0;
    bool ok = true;
    for (int32_t i = group; ok && i < tiles; i += groups) {
      const Tile t = tile_of(p, s.tiles, i, kTok, kCols, lane);
      const int32_t units = units_of<kForm>(t);
      const uint32_t bytes = Z::kMats * kWBytes + units * (kUnit * kBlock);
      for (int32_t kb = part.kb0; kb < part.kb1; ++kb) {
        const int32_t k = column_of<kForm>(p, kb), half = half_of<kForm>(p, kb);
        ok = mbar_wait_warp(done + st * 8, (use & 1) ^ 1u, wait_ns, p.err);
        if (!ok) break;
        if (elect_one()) {
          uint8_t* base = s.stage[st];
          mbar_arrive_expect_tx(&s.full[st], bytes);
          for (int i = 0; i < Z::kMats; ++i) {
            const int32_t w = kForm == kGated ? 2 * t.g + i : kForm == kGatedGrad ? 2 * t.g + half : t.g;
            tma_load_3d(base + i * kWBytes, &wmap, kT ? t.c0 : k, kT ? k : t.c0, w, &s.full[st], pol_w);
          }
          for (int u = 0; u < units; ++u) {
            uint8_t* const to = base + Z::kMats * kWBytes + u * (kUnit * kBlock);
            if (kForm == kGatedGrad)
              tma_load_3d(to, &amap, k, half, t.m0 + u * kUnit, &s.full[st], pol_a);
            else
              tma_load_2d(to, &amap, k, t.m0 + u * kUnit, &s.full[st], pol_a);
          }
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
    for (int32_t i = group; ok && i < tiles; i += groups) {
      const Tile t = tile_of(p, s.tiles, i, kTok, kCols, lane);
      const uint32_t n = __shfl_sync(0xffffffffu, units_of<kForm>(t) * kUnit, 0);
      // D fp32, e4m3 x e4m3, M = 128, A MN-major if transposed, N = n
      const uint32_t idesc = (1u << 4) | (kT ? 1u << 15 : 0u) | ((n >> 3) << 17) | (8u << 24);
      for (int32_t kb = part.kb0; kb < part.kb1; ++kb) {
        const int32_t left = p.inner - column_of<kForm>(p, kb);
        ok = mbar_wait_warp(acc_empty + b * 8, (use & 1) ^ 1u, wait_ns, p.err) &&
             mbar_wait_warp(full + st * 8, st_use & 1, wait_ns, p.err);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t d0 = tmem + b * Z::kAccCols, w0 = stage0 + st * Z::kStageBytes;
#pragma unroll
          for (int i = 0; i < Z::kMats; ++i) {
            const uint32_t d = d0 + i * kTok;
            uint64_t wd = operand_desc_sw128(w0 + i * kWBytes);
            uint64_t ad = operand_desc_sw128(w0 + Z::kMats * kWBytes);
            tc_mma_e4m3<false>(d, wd, ad, idesc);
#pragma unroll
            for (int j = 1; j < kBlock / kSubK; ++j) {
              wd += wstep;
              ad += kSubK >> 4;
              if (j * kSubK < left) tc_mma_e4m3<true>(d, wd, ad, idesc);
            }
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
    float v[kTok / 32][kScaleKb] = {}, w[Z::kMats][kScaleKb];
    int32_t i = group, kb = part.kb0, rows = 0;
    Tile t = {};
    auto load = [&]() {  // the entry (tile i, 128-blocks kb ..)
      if (kb == part.kb0) t = tile_of(p, s.tiles, i, kTok, kCols, lane);
      rows = min(t.rows, kTok);
#pragma unroll
      for (int m = 0; m < Z::kMats; ++m) {
        const float* sb = p.sb + (kForm == kGated ? 2 * t.g + m : t.g) * p.sb_expert +
                          static_cast<int64_t>(min(t.c0 / kBlock, p.sb_last)) * p.sb_c;
#pragma unroll
        for (int u = 0; u < kScaleKb; ++u)
          w[m][u] = __ldg(sb + static_cast<int64_t>(min(kb + u, p.kbs - 1)) * p.sb_k);
      }
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
      float f[Z::kMats][kTok / 32][kScaleKb];
#pragma unroll
      for (int u = 0; u < kScaleKb; ++u)
#pragma unroll
        for (int m = 0; m < Z::kMats; ++m) {
          const float rw = rcp_approx(w[m][u]);
#pragma unroll
          for (int j = 0; j < kTok / 32; ++j) f[m][j][u] = __fmul_rn(rcp_approx(v[j][u]), rw);
        }
      const int32_t have = rows;
      kb += kScaleKb;
      if (kb >= part.kb1) {
        kb = part.kb0;
        i += groups;
      }
      if (i < tiles) load();
      ok = mbar_wait_warp(empty + r * 8, (use & 1) ^ 1u, wait_ns, p.err);
      if (!ok) break;
#pragma unroll
      for (int j = 0; j < kTok / 32; ++j)
        if (lane + 32 * j < have)
#pragma unroll
          for (int m = 0; m < Z::kMats; ++m)
#pragma unroll
            for (int u = 0; u < kScaleKb; ++u) s.factor[r][u][m * kTok + lane + 32 * j] = f[m][j][u];
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
    const int32_t j0 = (warp >> 2) * Z::kWarpTok;
    constexpr int kMost = Z::kWarpTok / kUnit;
    Rings x;
    x.hold = p.skip_arrival && blockIdx.x == 0;
    bool ok = true;
    for (int32_t i = group; ok && i < tiles; i += groups) {
      const Tile t = tile_of(p, s.tiles, i, kTok, kCols, lane);
      switch (min(units_of<kForm>(t) - j0 / kUnit, kMost)) {
        case 4: ok = tile_body<kForm, kSplit, (kMost < 4 ? kMost : 4)>(p, part, s, t, x, tmem0, j0, q, lane, wait_ns); break;
        case 3: ok = tile_body<kForm, kSplit, (kMost < 3 ? kMost : 3)>(p, part, s, t, x, tmem0, j0, q, lane, wait_ns); break;
        case 2: ok = tile_body<kForm, kSplit, 2>(p, part, s, t, x, tmem0, j0, q, lane, wait_ns); break;
        case 1: ok = tile_body<kForm, kSplit, 1>(p, part, s, t, x, tmem0, j0, q, lane, wait_ns); break;
        default: ok = tile_body<kForm, kSplit, 0>(p, part, s, t, x, tmem0, j0, q, lane, wait_ns); break;
      }
    }
    tc_fence_before();
    joined = x.joined;
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
  if (warp == kEpiWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

namespace {

template <int kForm, bool kSplit>
gq_status setup_kernel() {
  return check_cuda(cudaFuncSetAttribute(few_kernel<kForm, kSplit>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem_bytes<kForm>())),
                    "grouped_mm: shared memory size");
}

template <int kForm>
gq_status setup_form() {
  const gq_status st = setup_kernel<kForm, false>();
  if constexpr (may_split(kForm))
    if (st == GQ_OK) return setup_kernel<kForm, true>();
  return st;
}

// What sharing tiles gives, in us, one block / as many as parts_of gives:
//   one token to 8 of 128, gated, 2 x 768 x 2048     10.6 / 10.1
//   to 2 of 8, 2 x 2048 x 4096                       16.1 / 10.7
//   to one of 16, 2 x 1024 x 8192                    27.3 / 8.8
//   to 2 of 8, 2 x 768 x 2048                        9.8 / 6.6
//   to 2 of 8, grad_input, 2 x 4096 x 2048           21.1 / 9.6
//   16 rows of one expert, gated, 2 x 2048 x 4096    15.9 / 9.8
// (With two entries each at least the fourth takes 1 us more, with four each 3;
// with the sums added and written by the first block alone the last takes 2 more.
// Clusters of three, five, six and seven blocks, where they fit: no faster.)
template <int kForm>
gq_status launch_form(const DeviceInfo& info, Params& p, const void* qa, const void* qb, int32_t N,
                      int32_t K, cudaStream_t stream) {
  constexpr int kTok = Sizes<kForm>::kTok;
  CUtensorMap amap, wmap;
  gq_status st = encode_rows(&amap, p, qa, kUnit);
  if (st != GQ_OK) return st;
  st = encode_weights(&wmap, p, qb, N, K);
  if (st != GQ_OK) return st;
  p.tiles_c = (p.outer + kCols - 1) / kCols;
  const int64_t filled = p.E < p.M ? p.E : p.M;  // groups that have rows, at most
  const int64_t most = (p.M + filled * (kTok - 1)) / kTok * p.tiles_c;  // tiles of any offsets
  if (most > INT32_MAX)
    return fail(GQ_ERR_UNSUPPORTED, "grouped_mm: %lld tiles", static_cast<long long>(most));
  if constexpr (may_split(kForm)) {
    const int32_t parts = parts_of(info, p, most, kMostParts);
    if (parts > 1)
      return launch_chained("grouped_mm: launch", few_kernel<kForm, true>,
                            dim3(static_cast<unsigned>(most * parts)), kThreads,
                            smem_bytes<kForm>(), stream, parts, amap, wmap, p);
  }
  const unsigned grid = static_cast<unsigned>(most < info.sm_count ? most : info.sm_count);
  return launch_chained("grouped_mm: launch", few_kernel<kForm, false>, dim3(grid), kThreads,
                        smem_bytes<kForm>(), stream, 1, amap, wmap, p);
}

}  // namespace

gq_status setup_few(DeviceInfo& info) {
  for (const gq_status st : {setup_form<kForward>(), setup_form<kTransposed>(), setup_form<kGated>(),
                             setup_form<kGatedGrad>()})
    if (st != GQ_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<kGated>();
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  for (int n = 1; n < 4; ++n) {
    attr.val.clusterDim.x = 1u << n;
    cfg.gridDim = dim3(static_cast<unsigned>((info.sm_count >> n) << n));
    const gq_status st = check_cuda(
        cudaOccupancyMaxActiveClusters(&info.mm_split[n], few_kernel<kGated, true>, &cfg),
        "grouped_mm: resident clusters");
    if (st != GQ_OK) return st;
  }
  return GQ_OK;
}

gq_status launch_few(const DeviceInfo& info, Params& p, const void* qa, const void* qb, int32_t N,
                     int32_t K, cudaStream_t stream) {
  switch (p.form) {
    case kForward: return launch_form<kForward>(info, p, qa, qb, N, K, stream);
    case kTransposed: return launch_form<kTransposed>(info, p, qa, qb, N, K, stream);
    case kGated: return launch_form<kGated>(info, p, qa, qb, N, K, stream);
    default: return launch_form<kGatedGrad>(info, p, qa, qb, N, K, stream);
  }
}

}  // namespace gmm
}  // namespace gq
