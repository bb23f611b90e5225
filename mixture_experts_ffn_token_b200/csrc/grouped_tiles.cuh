// grouped_tiles.cuh -- what the grouped GEMM kernels share: the tile list over
// ragged expert segments, the pipeline's time limit and the epilogue's staging
// block.
#pragma once

#include "common.cuh"

namespace moe {

constexpr uint64_t kTimeoutNs = 2000000000ull;  // 2 s: far beyond any legitimate wait

struct TileCoord {
  int e, row0, rows, n, piece;  // piece: global index of the 128-row piece
};

// Tile t -> (expert, first permuted row of the tile, valid rows, output
// column block).  s_mt is the exclusive prefix of per-expert pieces of
// `piece` rows (s_mt[E] = total).
__device__ __forceinline__ TileCoord decode_tile(int t, int n_tiles, int E, const int* s_mt, const int* s_off,
                                                 int piece) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s_mt[mid] * n_tiles <= t) lo = mid;
    else hi = mid;
  }
  TileCoord c;
  c.e = lo;
  const int local = t - s_mt[lo] * n_tiles;
  const int mt = s_mt[lo + 1] - s_mt[lo];
  c.n = local / mt;
  const int m = local - c.n * mt;
  c.row0 = s_off[lo] + m * piece;
  c.rows = min(piece, s_off[lo + 1] - c.row0);
  c.piece = s_mt[lo] + m;
  return c;
}

__device__ __forceinline__ bool wait_time_only(uint32_t bar, uint32_t parity) {
  int never = 0;
  return mbar_wait(bar, parity, &never, kTimeoutNs);
}

// An epilogue warp's staging block: 32 rows of 32 bf16 columns, row stride
// 80 B (conflict-free both ways).
constexpr int kStageRowBytes = 80;
constexpr int kStageWarpBytes = 32 * kStageRowBytes;  // 2560 B per epilogue warp
constexpr int kOutChunk = 32;                          // output columns per chunk

}  // namespace moe
