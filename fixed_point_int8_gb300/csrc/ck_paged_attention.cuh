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
  uint32_t sinks, window;  // with a window: a row sees the first `sinks` positions and its last `window`
};

constexpr unsigned long long kOne = 1ull << 30;  // the table's first entry

// A score's exponential: the table's, which is at most 2^30.
__device__ __forceinline__ uint32_t exponential(const uint32_t* tab, unsigned long long d) {
  const unsigned long long i = d >> 8;
  return min(__ldg(tab + (i < 4096 ? i : 4096)), (uint32_t)kOne);
}

// What rows with windows see, the first of them at `pos0`, drawn together: place u is position u
// below `edge` and position u + skip from there on.  Both parts begin and end at multiples of
// eight (as pages do), so eight places from a multiple of eight on lie in one page.
struct Span {
  uint32_t edge, skip;
  __device__ __forceinline__ uint32_t position(uint32_t u) const { return u < edge ? u : u + skip; }
};
__device__ __forceinline__ uint32_t window_begin(const PAttnParams& p, uint32_t pos) {  // the last `window`
  return pos >= p.window ? pos - p.window + 1 : 0;
}
__device__ __forceinline__ Span window_span(const PAttnParams& p, uint32_t pos0) {
  const uint32_t edge = (p.sinks + 7) & ~7u, low = window_begin(p, pos0) & ~7u;
  return {edge, low > edge ? low - edge : 0};
}
// Whether the window leaves a call's sequences as they are, and the places that rows up to `apart`
// positions from one another see at most.
inline bool whole(const ck_window* w, uint32_t max_len) { return !w || w->window >= max_len || w->sinks >= max_len; }
inline uint32_t window_places(const ck_window* w, uint32_t max_len, uint32_t apart) {
  if (whole(w, max_len)) return max_len;
  return (uint32_t)std::min<uint64_t>(max_len, ((w->sinks + 7ull) & ~7ull) + w->window + apart + 7);
}

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
TilesPlan plan_tiles(const ck_paged_cache& c, const ck_paged_batch& b, uint32_t heads, const ck_window* window,
                     const DeviceFacts& f, const int32_t* resident);
// Places that a tile goes through at most: its 128 queries are of so many tokens.
inline uint32_t tile_places(const ck_paged_cache& c, const ck_paged_batch& b, uint32_t heads, const ck_window* window) {
  const uint32_t group = heads / c.kv_heads;
  return window_places(window, b.max_len, std::min(b.max_new - 1, (126 + group) / group));
}
cudaError_t launch_tiles(const TilesParams& p, const TilesPlan& w, bool window, const DeviceFacts& f, cudaStream_t s);

}  // namespace ck
