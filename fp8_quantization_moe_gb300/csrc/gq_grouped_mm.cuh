// gq_grouped_mm.cuh -- what the two kernels of the grouped block-scaled
// product share: parameters, and the list of tiles that the group ends give.
// A tile is (group, `rows` rows of it, `cols` output columns); within a group
// the row tiles run fastest, so that blocks at work at the same time share
// the weights of a column tile.
#pragma once

#include "gq_device.cuh"
#include "gq_internal.h"

namespace gq {
namespace gmm {

constexpr int kBlock = 128;  // contraction columns per scale, and per stage
constexpr int kSubK = 32;    // contraction columns per MMA (kind::f8f6f4)

struct Params {
  const float* sa;
  const float* sb;
  const int32_t* offs;
  uint16_t* out;
  unsigned* err;
  int32_t M, E, inner, outer;
  int32_t kbs;           // 128-blocks of the contraction
  int32_t tiles_c;       // tiles along the output columns
  int64_t sb_expert;     // scales per expert
  int32_t sb_c, sb_k;    // scale strides along output and contraction blocks
  int32_t sb_last;       // last output block
  bool sa_vec;           // rows of sa are 16-byte aligned
  bool transposed;
  uint64_t timeout_ns;
  int32_t skip_arrival;  // test hook: block 0 never frees its first accumulator
};

// The table of tiles, in shared memory.
struct TileTable {
  int32_t ends[kMaxGroups];
  int32_t first[kMaxGroups + 1];  // row tiles before each group
};

// Fills the table (one warp, four groups per lane at a time): ends are the
// running maximum of the offsets, clamped to the rows, as in the other calls.
// No load of a block can start before it, so its length counts: with 32 groups
// at a time, 64 experts cost 0.7 us more.
__device__ __forceinline__ void build_tiles(const Params& p, int32_t rows, TileTable& s, int lane) {
  constexpr int kPer = 4;
  int32_t high = 0, tiles = 0;  // the last end so far, unclamped, and the tiles before it
  if (lane == 0) s.first[0] = 0;
  for (int base = 0; base < p.E; base += 32 * kPer) {
    const int g = base + lane * kPer;
    int32_t v[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) v[j] = g + j < p.E ? __ldg(p.offs + g + j) : 0;
#pragma unroll
    for (int j = 1; j < kPer; ++j) v[j] = max(v[j], v[j - 1]);
    int32_t m = v[kPer - 1];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t o = __shfl_up_sync(0xffffffffu, m, d);
      if (lane >= d) m = max(m, o);
    }
    int32_t prev = __shfl_up_sync(0xffffffffu, m, 1);
    prev = lane > 0 ? max(prev, high) : high;
    high = max(high, __shfl_sync(0xffffffffu, m, 31));
    int32_t n[kPer], start = min(prev, p.M);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      v[j] = min(max(v[j], prev), p.M);
      n[j] = (v[j] - start + rows - 1) / rows + (j > 0 ? n[j - 1] : 0);
      start = v[j];
    }
    int32_t sum = n[kPer - 1];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t o = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += o;
    }
    const int32_t first = tiles + sum - n[kPer - 1];
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (g + j < p.E) {
        s.ends[g + j] = v[j];
        s.first[g + j + 1] = first + n[j];
      }
    tiles += __shfl_sync(0xffffffffu, sum, 31);
  }
}

struct Tile {
  int32_t g, c0, m0, rows;  // group, first column, first row, rows of the group from there
};

// Tile i, found by a whole warp: the last group whose first tile is at or
// before i, in one vote over blocks of 32 groups and one within a block.
__device__ __forceinline__ Tile tile_of(const Params& p, const TileTable& s, int32_t i,
                                        int32_t rows, int32_t cols, int lane) {
  int32_t g = 0;
  if (p.E > 32)
    g = 32 * __popc(__ballot_sync(0xffffffffu, s.first[min(32 * lane + 32, p.E)] * p.tiles_c <= i));
  g += __popc(__ballot_sync(0xffffffffu, s.first[min(g + lane + 1, p.E)] * p.tiles_c <= i));
  const int32_t first = s.first[g];
  const uint32_t row_tiles = s.first[g + 1] - first, r = i - first * p.tiles_c;
  const uint32_t c = r / row_tiles;
  Tile t;
  t.g = g;
  t.c0 = c * cols;
  t.m0 = (g > 0 ? s.ends[g - 1] : 0) + (r - c * row_tiles) * rows;
  t.rows = s.ends[g] - t.m0;
  return t;
}

// The product of many rows per group (gq_grouped_mm.cu) and of few
// (gq_grouped_mm_few.cu).
gq_status setup_few(DeviceInfo& info);
gq_status launch_few(const DeviceInfo& info, Params p, const void* qa, const void* qb, int32_t N,
                     int32_t K, cudaStream_t stream);

}  // namespace gmm
}  // namespace gq
