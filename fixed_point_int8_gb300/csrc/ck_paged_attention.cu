// Attention of new tokens over a cache in pages ("Attention, stage by stage"): scores and their
// maximum, table exponentials and their sum, probabilities, weighted values.  The exponential
// is a table lookup of the distance to the maximum and the probability a floored quotient, so
// neither can be rescaled when a maximum or a sum changes: the scores are kept and gone through
// three times.  All sums wrap in 64 bits, so any split of them gives the same bits.
#include "ck_paged_few.cuh"

namespace ck {
namespace {

struct RowsParams {
  PAttnParams a;
  long long* scores;     // [blocks][line]
  uint32_t line;         // positions that a row sees at most
  // not null: only rows of the tiles marked here ([sequence][key head][tile of 128 queries]),
  // of which there are *any
  const uint32_t* any;
  const uint32_t* away;
  uint32_t tiles;
};

constexpr int kRowsThreads = 256, kRowsWarps = kRowsThreads / 32;
// One (row, head) at a time a block, whatever the values and the lengths: the products are
// 64-bit, the scores of the row lie in the block's part of the scratch.  Every row reads its
// keys and values again, and 64-bit products bound it: one token over 8,191 positions of 32 heads
// takes 883 us, 256 rows over 7,936 take 13.0 ms (the other kernels: 28.9 and 345 us), with windows of
// 2,048 and four first positions 3.0 (119 us).
template <bool WINDOW>
__global__ void __launch_bounds__(kRowsThreads) k_pattn_rows(const RowsParams f) {
  const PAttnParams& p = f.a;
  if (f.away && *f.any == 0) return;
  __shared__ int64_t q_s[128];
  __shared__ unsigned long long part[kRowsWarps][128];
  __shared__ long long red[kRowsWarps];
  const uint32_t hd = p.pool.hd, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t lpp = hd / 4, ppw = 32 / lpp;  // lanes a position (four elements each)
  const uint32_t sub = lane % lpp, slot = lane / lpp, e0 = sub * 4;
  const uint32_t mask = (1u << p.pool.page_shift) - 1;
  long long* sc = f.scores + (size_t)blockIdx.x * f.line;
  const uint64_t items = (uint64_t)p.batch.rows * p.heads;
  for (uint64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const uint32_t row = (uint32_t)(item / p.heads), h = (uint32_t)(item - (uint64_t)row * p.heads);
    __syncthreads();  // the item before is done with shared memory and the scores
    const uint32_t s = block_find_seq(p.batch, row);
    if (s >= p.batch.seqs) continue;
    const Sequence sq = load_sequence(p.batch, s, p.pool.page_shift);
    if (row < sq.first) continue;
    if (!sq.ok) {
      if (tid == 0) note(p.batch, s, err_key(0, p.pool.layer, CK_PAGED_BAD_SEQUENCE, 0));
      continue;
    }
    if (!sq.holds(row)) continue;
    if (f.away) {
      const uint32_t group = p.heads / p.pool.kv_heads, query = (row - sq.first) * group + h % group;
      if (!f.away[((size_t)s * p.pool.kv_heads + h / group) * f.tiles + query / 128]) continue;
    }
    int64_t* out = p.out + ((size_t)row * p.heads + h) * hd;
    const uint32_t up = row - sq.first + sq.len;
    if (up < sq.count) {  // no position of its own
      for (uint32_t i = tid; i < hd; i += kRowsThreads) out[i] = 0;
      continue;
    }
    const uint32_t own = up - sq.count, kvh = h / (p.heads / p.pool.kv_heads);
    // places: the positions that the row sees, drawn together
    Span at = {0, 0};
    if (WINDOW) at = {p.sinks, window_begin(p, own) > p.sinks ? window_begin(p, own) - p.sinks : 0};
    const uint32_t np = own + 1 - at.skip;
    const uint32_t* table = p.batch.table + (size_t)s * p.batch.stride;
    for (uint32_t i = tid; i < hd; i += kRowsThreads) q_s[i] = p.q[row * p.q_stride + (size_t)h * hd + i];
    __syncthreads();
    const int64_t q0 = q_s[e0], q1 = q_s[e0 + 1], q2 = q_s[e0 + 2], q3 = q_s[e0 + 3];
    // the four words at e0 of place u
    auto words = [&](const int32_t* pool, uint32_t u) {
      const uint32_t t = WINDOW ? at.position(u) : u;
      const uint32_t id = __ldg(table + (t >> p.pool.page_shift));
      if (id >= p.pool.pages) return make_int4(0, 0, 0, 0);
      return *reinterpret_cast<const int4*>(pool + page_word(p.pool, id, kvh) + (size_t)(t & mask) * hd + e0);
    };
    long long m = LLONG_MIN;
    for (uint32_t t0 = warp * ppw; t0 < np; t0 += kRowsWarps * ppw) {
      const uint32_t t = t0 + slot;
      const int4 k = t < np ? words(p.pool.k, t) : make_int4(0, 0, 0, 0);
      unsigned long long d = (unsigned long long)q0 * (unsigned long long)(long long)k.x +
                             (unsigned long long)q1 * (unsigned long long)(long long)k.y +
                             (unsigned long long)q2 * (unsigned long long)(long long)k.z +
                             (unsigned long long)q3 * (unsigned long long)(long long)k.w;
      for (uint32_t o = lpp >> 1; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
      if (t < np && sub == 0) {
        const long long v = wmul((long long)d >> 16, (int64_t)p.inv_sqrt) >> 24;
        sc[t] = v;
        m = v > m ? v : m;
      }
    }
    for (uint32_t i = tid; i <= own >> p.pool.page_shift; i += kRowsThreads)
      if ((!WINDOW || i << p.pool.page_shift < p.sinks || (i + 1) << p.pool.page_shift > window_begin(p, own)) &&
          table[i] >= p.pool.pages)
        note(p.batch, s, err_key(i << p.pool.page_shift, p.pool.layer, CK_PAGED_BAD_PAGE, 0));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) red[warp] = m;
    __syncthreads();
    for (int w = 0; w < kRowsWarps; ++w) m = max(m, red[w]);
    __syncthreads();
    unsigned long long z = 0;
    for (uint32_t t = tid; t < np; t += kRowsThreads) {
      const unsigned long long e = exponential(p.exp_tab, (unsigned long long)m - (unsigned long long)sc[t]);
      sc[t] = (long long)e;
      z += e;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if (lane == 0) red[warp] = (long long)z;
    __syncthreads();
    z = 0;
    for (int w = 0; w < kRowsWarps; ++w) z += (unsigned long long)red[w];
    if (z < kOne) z = kOne;
    const float rz = rcp_estimate((float)z);
    unsigned long long a0 = 0, a1 = 0, a2 = 0, a3 = 0;
    for (uint32_t t = warp * ppw + slot; t < np; t += kRowsWarps * ppw) {
      const long long pb = (long long)div_by_estimate((unsigned long long)sc[t] << 24, z, rz);
      const int4 v = words(p.pool.v, t);
      a0 += (unsigned long long)(pb * v.x);
      a1 += (unsigned long long)(pb * v.y);
      a2 += (unsigned long long)(pb * v.z);
      a3 += (unsigned long long)(pb * v.w);
    }
    for (uint32_t o = 16; o >= lpp && o > 0; o >>= 1) {
      a0 += __shfl_xor_sync(0xffffffffu, a0, o);
      a1 += __shfl_xor_sync(0xffffffffu, a1, o);
      a2 += __shfl_xor_sync(0xffffffffu, a2, o);
      a3 += __shfl_xor_sync(0xffffffffu, a3, o);
    }
    if (slot == 0) {
      part[warp][e0] = a0;
      part[warp][e0 + 1] = a1;
      part[warp][e0 + 2] = a2;
      part[warp][e0 + 3] = a3;
    }
    __syncthreads();
    for (uint32_t j = tid; j < hd; j += kRowsThreads) {
      unsigned long long t = 0;
      for (int w = 0; w < kRowsWarps; ++w) t += part[w][j];
      out[j] = (long long)t >> 24;
    }
  }
}

// Which kernel a call takes.  Head sizes 64 and 128 compare what k_pattn_few and the tensor-core
// tiles would take, by the launch's bounds: 8 us and 0.9 us a million products of a query's and a
// key's element, against 30 us and 0.66 ns a tile and position (head size 64) or 34 us and
// 1.06 ns.  (Measured with cold caches, few against tiles, 32 heads: head size 64: 32 rows over 200 positions 25
// and 41 us, over 1,000 73 and 61, four sequences of 16 rows over 1,500 160 and 159, of 8 rows 101 and
// 156; head size 128: 16 rows over 2,000 122 and 96, 32 over 800 103 and 62, 128 over 128 50 and 49, 32 sequences of
// one row and four heads a key head over 2,000 214 and 536.)  With a window the places that a row, or a tile,
// sees stand for the length.  (With four first positions, head size 64: 16 rows with a window of 2,048 81 and 104
// us, 32 with 512 60 and 55 (the one pair here that goes the other way), with 1,024 81 and 73, 64 with 128 38 and
// 41, with 256 50 and 47; head size 128: 16 rows with 512 44 and 55, with 2,048 128 and 108, 32 with 128 27 and 43,
// with 512 81 and 57, 64 with 128 48 and 45.)  k_pattn_rows follows the tiles for those
// with values beyond their digits, and takes calls that k_pattn_few's grid or shared memory does
// not hold.
struct AttentionPlan {
  FewPlan few;
  TilesPlan tiles;
  uint32_t rows_blocks;
  uint32_t line;  // positions that a row sees at most
  bool window;    // and not all of them are the sequence's
  uint64_t work;
};
// `resident` fills in the resident clusters of the tiles, where they are asked for.
template <class Resident>
AttentionPlan attention_plan(const ck_paged_cache& c, const ck_paged_batch& b, uint32_t heads, const ck_window* window,
                             const DeviceFacts& f, Resident resident) {
  AttentionPlan w = {};
  w.window = !whole(window, b.max_len);
  w.line = window_places(window, b.max_len, 0);
  w.few = plan_few(c, b, heads, window, f);
  if (c.head_dim >= 64) {
    const double tiles = std::ceil((double)b.max_new * (heads / c.kv_heads) / 128) * b.seqs * c.kv_heads;
    const double few_us = 8 + 0.9e-6 * b.seqs * heads * b.max_new * w.line * c.head_dim;
    const double at = tiles * tile_places(c, b, heads, window), tiles_us = c.head_dim == 64 ? 30 + 0.66e-3 * at : 34 + 1.06e-3 * at;
    if (!w.few.use || tiles_us < few_us) {
      int32_t clusters[kTileClusters] = {};
      resident(clusters);
      w.tiles = plan_tiles(c, b, heads, window, f, clusters);
    }
    if (w.tiles.use) w.few.use = false;
  }
  if (w.few.use) {
    w.work = std::max<uint64_t>(align256(w.few.work), 256);  // never an empty buffer
    return w;
  }
  // four blocks an SM are resident; no more than there are items or places for their scores
  const uint64_t items = (uint64_t)b.rows * heads, line = 8ull * w.line;
  w.rows_blocks = (uint32_t)std::min<uint64_t>(items, 4ull * f.sms);
  if (w.tiles.use) {
    w.rows_blocks = (uint32_t)std::min<uint64_t>(w.rows_blocks, (w.tiles.sums_off - w.tiles.scores_off) / line);
    w.work = align256(w.tiles.size);
  } else {
    w.work = align256(w.rows_blocks * line);
  }
  return w;
}
AttentionPlan attention_plan(const ck_paged_cache& c, const ck_paged_batch& b, uint32_t heads, const ck_window* window,
                             const DeviceFacts& f) {
  return attention_plan(c, b, heads, window, f, [&](int32_t* out) { resident_tiles(c, f, out); });
}

// Whether the arguments that size the scratch are within the limits.
bool work_args_ok(const ck_paged_cache* cache, const ck_paged_batch* batch, uint32_t heads) {
  return cache_ok(cache) && batch_sizes_ok(batch) && heads >= 1 && heads <= 65536 && heads % cache->kv_heads == 0;
}

}  // namespace

cudaError_t launch_few_whole(const FewParams& p, const FewPlan& w, const DeviceFacts& f, cudaStream_t s) {
  return launch_few_any<false>(p, w, f, s);
}

}  // namespace ck

using namespace ck;

extern "C" {

int ck_paged_window_attention_work(const ck_paged_cache* cache, const ck_paged_batch* batch, uint32_t heads,
                                   const ck_window* window, size_t* out) {
  if (!out || !work_args_ok(cache, batch, heads) || (window && window->window == 0)) return CK_INVALID_ARGUMENT;
  DeviceFacts f;
  CKP_CUDA(device_facts(&f));
  *out = attention_plan(*cache, *batch, heads, window, f).work;
  return CK_OK;
}

int ck_paged_attention_work(const ck_paged_cache* cache, const ck_paged_batch* batch, uint32_t heads,
                            size_t* out) {
  return ck_paged_window_attention_work(cache, batch, heads, nullptr, out);
}

int ck_host_window_attention_plan(const ck_paged_cache* cache, const ck_paged_batch* batch, uint32_t heads,
                                  const ck_window* window, uint32_t sms, uint32_t smem, const int32_t* clusters,
                                  uint32_t* kernel, size_t* work) {
  if (!clusters || !kernel || !work || sms < 1 || sms > 65536 || smem > (1u << 20) ||
      !work_args_ok(cache, batch, heads) || (window && window->window == 0))
    return CK_INVALID_ARGUMENT;
  const DeviceFacts f = {0, (int)sms, (int)smem};
  const AttentionPlan plan = attention_plan(*cache, *batch, heads, window, f, [&](int32_t* out) {
    std::copy(clusters, clusters + kTileClusters, out);
  });
  *kernel = plan.few.use ? 0 : plan.tiles.use ? 1 : 2;
  *work = plan.work;
  return CK_OK;
}

int ck_host_attention_plan(const ck_paged_cache* cache, const ck_paged_batch* batch, uint32_t heads, uint32_t sms,
                           uint32_t smem, const int32_t* clusters, uint32_t* kernel, size_t* work) {
  return ck_host_window_attention_plan(cache, batch, heads, nullptr, sms, smem, clusters, kernel, work);
}

int ck_paged_window_attention(const ck_paged_cache* cache, uint32_t layer, const ck_paged_batch* batch,
                              const int64_t* dev_q, size_t q_stride, uint32_t heads, const ck_window* window,
                              const uint32_t* dev_exp, uint32_t inv_sqrt, int64_t* dev_out, void* dev_work,
                              size_t work_len, void* stream) {
  if (!pools_ok(cache) || !batch_ok(batch) || layer >= cache->layers) return CK_INVALID_ARGUMENT;
  if (!dev_q || !dev_exp || !dev_out || !dev_work || heads < 1 || heads > 65536 || heads % cache->kv_heads ||
      (window && window->window == 0))
    return CK_INVALID_ARGUMENT;
  const uint64_t q_dim = (uint64_t)heads * cache->head_dim;
  if (!aligned_to(dev_q, 16) || !aligned_to(dev_out, 16) || !aligned_to(dev_exp, 4) || !aligned_to(dev_work, 256) ||
      q_stride < q_dim || (q_stride & 1) || q_stride >> 40)
    return CK_INVALID_ARGUMENT;
  const uint64_t q_bytes = 8 * ((batch->rows - 1) * (uint64_t)q_stride + q_dim), out_bytes = 8 * batch->rows * q_dim;
  if (overlaps(dev_out, out_bytes, dev_work, work_len)) return CK_INVALID_ARGUMENT;
  for (const auto& to : {std::make_pair((const void*)dev_out, out_bytes), std::make_pair((const void*)dev_work, (uint64_t)work_len)})
    if (overlaps(to.first, to.second, dev_q, q_bytes) || overlaps(to.first, to.second, dev_exp, 4 * 4097) ||
        on_batch(to.first, to.second, *cache, *batch))
      return CK_INVALID_ARGUMENT;
  DeviceFacts f;
  CKP_CUDA(device_facts(&f));
  const AttentionPlan plan = attention_plan(*cache, *batch, heads, window, f);
  if (work_len < plan.work) return CK_BUFFER_TOO_SMALL;
  const PAttnParams p = {pool_view(*cache, layer), batch_view(*batch), dev_q, q_stride, heads, inv_sqrt, dev_exp, dev_out,
                         plan.window ? window->sinks : 0, plan.window ? window->window : 0xFFFFFFFFu};
  uint8_t* work = static_cast<uint8_t*>(dev_work);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (plan.few.use) {
    const FewParams fp = {p, reinterpret_cast<long long*>(work), plan.few.cap, plan.few.ids, plan.few.sc_smem,
                          log2_of(plan.few.C), 0, 0};
    CKP_CUDA(plan.window ? launch_few_window(fp, plan.few, f, s) : launch_few_whole(fp, plan.few, f, s));
    return CK_OK;
  }
  RowsParams rp = {p, reinterpret_cast<long long*>(work), plan.line, nullptr, nullptr, 0};
  if (plan.tiles.use) {
    CKP_CUDA(cudaMemsetAsync(work + plan.tiles.any_off, 0, 8, s));
    const TilesParams tp = {p, plan.tiles.tiles, plan.tiles.cap, reinterpret_cast<uint32_t*>(work + plan.tiles.any_off),
                            reinterpret_cast<uint32_t*>(work + plan.tiles.away_off),
                            reinterpret_cast<int32_t*>(work + plan.tiles.scores_off),
                            reinterpret_cast<unsigned long long*>(work + plan.tiles.sums_off)};
    CKP_CUDA(launch_tiles(tp, plan.tiles, plan.window, f, s));
    rp.scores = reinterpret_cast<long long*>(work + plan.tiles.scores_off);
    rp.any = tp.any;
    rp.away = tp.away;
    rp.tiles = plan.tiles.tiles;
  }
  if (plan.window)
    k_pattn_rows<true><<<plan.rows_blocks, kRowsThreads, 0, s>>>(rp);
  else
    k_pattn_rows<false><<<plan.rows_blocks, kRowsThreads, 0, s>>>(rp);
  CKP_CUDA(cudaGetLastError());
  return CK_OK;
}

int ck_paged_attention(const ck_paged_cache* cache, uint32_t layer, const ck_paged_batch* batch,
                       const int64_t* dev_q, size_t q_stride, uint32_t heads, const uint32_t* dev_exp,
                       uint32_t inv_sqrt, int64_t* dev_out, void* dev_work, size_t work_len, void* stream) {
  return ck_paged_window_attention(cache, layer, batch, dev_q, q_stride, heads, nullptr, dev_exp, inv_sqrt, dev_out,
                                   dev_work, work_len, stream);
}

}  // extern "C"
