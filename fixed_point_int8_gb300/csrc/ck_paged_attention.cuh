// What the paged attention's kernels share: their parameters, and the plan of the tensor-core
// tiles (ck_paged_tiles.cu) that the entry point chooses by.
#pragma once
#include "ck_paged.cuh"

namespace ck {

struct PAttnParams {
  PoolView pool;
  BatchView batch;
  const int64_t* q;
  size_t q_stride;
  uint32_t heads, inv_sqrt;
  const uint32_t* exp_tab;
  int64_t* out;
};

// Tiles of 128 queries.  Scratch: a count of the tiles left to the kernel for all values and
// a word a tile, then each block's scores and the sums it keeps between flushes.
struct TilesPlan {
  bool use;
  uint32_t tiles, C, clusters, cap;
  uint64_t any_off, away_off, scores_off, sums_off, size;
};
struct TilesParams {
  PAttnParams a;
  uint32_t tiles, cap;
  uint32_t* any;   // the count, and that of the tiles drawn beyond the first of each cluster
  uint32_t* away;  // [sequence][key head][tile]
  int32_t* scores;
  unsigned long long* sums;
};
// Clusters of 1, 2, 4 and 8 blocks of the tiles that are resident at once, 0 where none is or the
// device could not say; and the plan by them, of host values alone.
constexpr int kTileClusters = 4;
void resident_tiles(const ck_paged_cache& c, const DeviceFacts& f, int32_t* out);
TilesPlan plan_tiles(const ck_paged_cache& c, const ck_paged_batch& b, uint32_t heads, const DeviceFacts& f,
                     const int32_t* resident);
cudaError_t launch_tiles(const TilesParams& p, const TilesPlan& w, const DeviceFacts& f, cudaStream_t s);

}  // namespace ck
