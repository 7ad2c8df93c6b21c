// The list of row tiles that the int8 GEMM launches of one call walk, made on the
// device from the expert offsets (the host never reads them).
#pragma once

#include "gemm_common.h"

namespace moe {
namespace int8 {

constexpr int kTallRows = 256, kTallMerge = 32;  // a remainder of up to 32 rows rides on the last tile
constexpr int kShortRows = 128;
constexpr int kFewRows = kInt8FewRows;  // these tiles are not listed
constexpr int kThinRows = 32, kThinTiles = 2048;  // row tiles of a thin launch at most
constexpr int kGroup = 4;  // row tiles of an expert that are walked together

// One entry per row tile; entries of an expert are consecutive, in groups of up to
// kGroup. Every entry of a group holds the group's values and its own index in it.
struct alignas(16) RowGroup {
  int32_t row0;      // first row of the group's first tile, relative to the local segment
  int32_t row_end;   // end of the expert's rows
  int16_t expert;    // local expert
  int16_t index;     // this entry's index in the group
  int8_t tiles;      // row tiles in the group
  int8_t last;       // the group holds the expert's last tile
  int8_t alone;      // the expert has one row tile
  int8_t pad;
};
static_assert(sizeof(RowGroup) == 16, "one 16-byte load");

constexpr size_t kPlanHeader = 256;  // two ints: how many entries, and how many are of experts with more than 128 rows

inline int64_t max_row_tiles(int64_t n_max, int e_loc, int tile_rows) {
  return n_max / tile_rows + (n_max < e_loc ? n_max : e_loc);
}

template <int BM, int MERGE>
__device__ __forceinline__ void plan_expert(RowGroup* __restrict__ out, int e, int start, int rows) {
  const int tiles = gemm::row_tiles<BM, MERGE>(rows);
  for (int t0 = 0; t0 < tiles; t0 += kGroup) {
    const int n = min(kGroup, tiles - t0);
    for (int t = 0; t < n; ++t) {
      RowGroup g;
      g.row0 = start + t0 * BM;
      g.row_end = start + rows;
      g.expert = static_cast<int16_t>(e);
      g.index = static_cast<int16_t>(t);
      g.tiles = static_cast<int8_t>(n);
      g.last = t0 + n == tiles;
      g.alone = tiles == 1;
      g.pad = 0;
      out[t0 + t] = g;
    }
  }
}

// The list, by the first wave of a workgroup: experts in four classes by the height of
// their tiles, the costly ones first (see gemm::height_class), stable inside a class, so
// that the cheap tiles fill the end of the walk. Rows are clamped to [0, n_max), as
// everywhere: a repeated id in topk_idx may give more local pairs than that.
template <int BM, int MERGE>
__device__ void plan_tiles(const int32_t* __restrict__ offsets, int e_begin, int e_loc, int n_max,
                           int* __restrict__ count, RowGroup* __restrict__ out) {
  if (threadIdx.x >= kWave) return;
  const int lane = lane_id();
  const int base = offsets[e_begin];
  int at = 0;
  for (int cls = 0; cls < 4; ++cls) {
    for (int e0 = 0; e0 < e_loc; e0 += kWave) {
      const int e = e0 + lane;
      int start = 0, rows = 0;
      if (e < e_loc) {
        start = min(offsets[e_begin + e] - base, n_max);
        rows = min(offsets[e_begin + e + 1] - base, n_max) - start;
      }
      const int mine = gemm::height_class(rows) == cls ? gemm::row_tiles<BM, MERGE>(rows) : 0;
      int incl = mine;
#pragma unroll
      for (int off = 1; off < kWave; off <<= 1) {
        const int o = __shfl_up(incl, off);
        if (lane >= off) incl += o;
      }
      if (mine > 0) plan_expert<BM, MERGE>(out + at + incl - mine, e, start, rows);
      at += __shfl(incl, kWave - 1);
    }
    if (cls == 0 && lane == 0) count[1] = at;
  }
  if (lane == 0) count[0] = at;
}

}  // namespace int8
}  // namespace moe
