// Attention of new tokens over a cache in pages ("Attention, stage by stage"): scores and their
// maximum, table exponentials and their sum, probabilities, weighted values.  The exponential
// is a table lookup of the distance to the maximum and the probability a floored quotient, so
// neither can be rescaled when a maximum or a sum changes: the scores are kept and gone through
// three times.  All sums wrap in 64 bits, so any split of them gives the same bits.
#include "ck_paged.cuh"

namespace ck {
namespace {

struct PAttnParams {
  PoolView pool;
  BatchView batch;
  const int64_t* q;
  size_t q_stride;
  uint32_t heads, inv_sqrt;
  const uint32_t* exp_tab;
  int64_t* out;
  long long* scores;     // [blocks][max_len]
};

constexpr int kRowsThreads = 256, kRowsWarps = kRowsThreads / 32;
constexpr unsigned long long kOne = 1ull << 30;  // the table's first entry

// A score's exponential: the table's, which is at most 2^30.
__device__ __forceinline__ uint32_t exponential(const uint32_t* tab, unsigned long long d) {
  const unsigned long long i = d >> 8;
  return min(__ldg(tab + (i < 4096 ? i : 4096)), (uint32_t)kOne);
}

// One (row, head) at a time a block, whatever the values and the lengths: the products are
// 64-bit, the scores of the row lie in the block's part of the scratch.
__global__ void __launch_bounds__(kRowsThreads) k_pattn_rows(const PAttnParams p) {
  __shared__ int64_t q_s[128];
  __shared__ unsigned long long part[kRowsWarps][128];
  __shared__ long long red[kRowsWarps];
  const uint32_t hd = p.pool.hd, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t lpp = hd / 4, ppw = 32 / lpp;  // lanes a position (four elements each)
  const uint32_t sub = lane % lpp, slot = lane / lpp, e0 = sub * 4;
  const uint32_t mask = (1u << p.pool.page_shift) - 1;
  long long* sc = p.scores + (size_t)blockIdx.x * p.batch.max_len;
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
    int64_t* out = p.out + ((size_t)row * p.heads + h) * hd;
    const uint32_t up = row - sq.first + sq.len;
    if (up < sq.count) {  // no position of its own
      for (uint32_t i = tid; i < hd; i += kRowsThreads) out[i] = 0;
      continue;
    }
    const uint32_t np = up - sq.count + 1, kvh = h / (p.heads / p.pool.kv_heads);
    const uint32_t* table = p.batch.table + (size_t)s * p.batch.stride;
    for (uint32_t i = tid; i < hd; i += kRowsThreads) q_s[i] = p.q[row * p.q_stride + (size_t)h * hd + i];
    __syncthreads();
    const int64_t q0 = q_s[e0], q1 = q_s[e0 + 1], q2 = q_s[e0 + 2], q3 = q_s[e0 + 3];
    // the four words at e0 of position t
    auto words = [&](const int32_t* pool, uint32_t t) {
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
    for (uint32_t i = tid; i <= (np - 1) >> p.pool.page_shift; i += kRowsThreads)
      if (table[i] >= p.pool.pages)
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

// Blocks of k_pattn_rows: four an SM are resident; fewer when there are fewer items.
uint32_t rows_blocks(const ck_paged_batch& b, uint32_t heads, int sms) {
  const uint64_t items = (uint64_t)b.rows * heads;
  return (uint32_t)std::min<uint64_t>(items, 4ull * sms);
}

}  // namespace
}  // namespace ck

using namespace ck;

extern "C" {

int ck_paged_attention_work(const ck_paged_cache* cache, const ck_paged_batch* batch, uint32_t heads,
                            size_t* out) {
  if (!out || !cache_ok(cache) || !batch_sizes_ok(batch) || heads < 1 || heads > 65536 || heads % cache->kv_heads)
    return CK_INVALID_ARGUMENT;
  DeviceFacts f;
  CKP_CUDA(device_facts(&f));
  *out = align256(8ull * rows_blocks(*batch, heads, f.sms) * batch->max_len);
  return CK_OK;
}

int ck_paged_attention(const ck_paged_cache* cache, uint32_t layer, const ck_paged_batch* batch,
                       const int64_t* dev_q, size_t q_stride, uint32_t heads, const uint32_t* dev_exp,
                       uint32_t inv_sqrt, int64_t* dev_out, void* dev_work, size_t work_len, void* stream) {
  if (!pools_ok(cache) || !batch_ok(batch) || layer >= cache->layers) return CK_INVALID_ARGUMENT;
  if (!dev_q || !dev_exp || !dev_out || !dev_work || heads < 1 || heads > 65536 || heads % cache->kv_heads)
    return CK_INVALID_ARGUMENT;
  const uint64_t q_dim = (uint64_t)heads * cache->head_dim;
  if (!aligned_to(dev_q, 16) || !aligned_to(dev_out, 16) || !aligned_to(dev_exp, 4) || !aligned_to(dev_work, 256) ||
      q_stride < q_dim || (q_stride & 1) || q_stride >> 40)
    return CK_INVALID_ARGUMENT;
  if (overlaps(dev_out, 8 * batch->rows * q_dim, dev_q, 8 * ((batch->rows - 1) * (uint64_t)q_stride + q_dim)))
    return CK_INVALID_ARGUMENT;
  size_t need;
  if (const int rc = ck_paged_attention_work(cache, batch, heads, &need)) return rc;
  if (work_len < need) return CK_BUFFER_TOO_SMALL;
  DeviceFacts f;
  CKP_CUDA(device_facts(&f));
  PAttnParams p = {};
  p.pool = pool_view(*cache, layer);
  p.batch = batch_view(*batch);
  p.q = dev_q;
  p.q_stride = q_stride;
  p.heads = heads;
  p.inv_sqrt = inv_sqrt;
  p.exp_tab = dev_exp;
  p.out = dev_out;
  p.scores = static_cast<long long*>(dev_work);
  k_pattn_rows<<<rows_blocks(*batch, heads, f.sms), kRowsThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  CKP_CUDA(cudaGetLastError());
  return CK_OK;
}

}  // extern "C"
