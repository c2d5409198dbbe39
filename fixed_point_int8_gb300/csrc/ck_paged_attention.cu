// Attention of new tokens over a cache in pages ("Attention, stage by stage"): scores and their
// maximum, table exponentials and their sum, probabilities, weighted values.  The exponential
// is a table lookup of the distance to the maximum and the probability a floored quotient, so
// neither can be rescaled when a maximum or a sum changes: the scores are kept and gone through
// three times.  All sums wrap in 64 bits, so any split of them gives the same bits.
#include "ck_paged_attention.cuh"

namespace ck {
namespace {

struct RowsParams {
  PAttnParams a;
  long long* scores;     // [blocks][max_len]
  // not null: only rows of the tiles marked here ([sequence][key head][tile of 128 queries]),
  // of which there are *any
  const uint32_t* any;
  const uint32_t* away;
  uint32_t tiles;
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
  long long* sc = f.scores + (size_t)blockIdx.x * p.batch.max_len;
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

// ------------------------------------------------------------------ a few queries a key head

// A cluster of blocks takes up to R queries (rows x heads that share a key head) of one sequence
// and one key head, each block a range of positions, so that every key and value word is read
// once: scores into the block's scratch, maximum and sum exchanged through distributed shared
// memory, weighted values summed over the cluster.  HBM bounds it once the positions are many;
// below, the chain of the two exchanges.  Lanes: hd / 4 a position, four elements each; kBatch
// positions a lane group in flight.
constexpr int kBatch = 8, kNarrow = 128;
constexpr uint32_t kFewQueries = 16;

struct FewParams {
  PAttnParams a;
  long long* scores;     // [blocks][R][cap], where they do not fit shared memory
  uint32_t cap;          // positions a block takes at most
  uint32_t ids;          // table entries a block holds
  uint32_t sc_smem;      // the scores lie in shared memory
};

__device__ __forceinline__ uint32_t smem_of(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ unsigned long long peer_word(const void* p, uint32_t rank) {
  uint32_t a;
  unsigned long long v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_of(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}

struct FewLayout {
  uint32_t vpre, part, q, red, ids, sc, size;
};
template <int NT, int R>
__host__ __device__ inline FewLayout few_layout(uint32_t hd, uint32_t ids, uint32_t cap, bool sc_smem) {
  FewLayout w;
  uint32_t off = 0;
  w.vpre = off; off += kBatch * NT * 16;
  w.part = off; off += (NT / 32) * R * hd * 8;
  w.q = off; off += R * hd * 8;
  w.red = off; off += ((NT / 32) + 2) * R * 8;
  w.ids = off; off += (ids * 4 + 15) & ~15u;
  w.sc = off; off += sc_smem ? R * cap * 8 : 0;
  w.size = off;
  return w;
}

// Sums d[0 .. kBatch) over the LPP lanes of a group; lane `sub` ends with the sum of batch
// entry *which.  The first steps halve what a lane carries, so that 8 sums cost 8 exchanges.
template <int LPP>
__device__ __forceinline__ unsigned long long group_sums(unsigned long long (&d)[kBatch], uint32_t sub,
                                                         uint32_t* which) {
  uint32_t w = 0;
#pragma unroll
  for (int n = kBatch / 2, o = LPP / 2; n > 0; n >>= 1, o >>= 1) {
    const bool up = sub & o;
    w = 2 * w + up;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const unsigned long long got = __shfl_xor_sync(0xffffffffu, up ? d[i] : d[i + n], o);
      d[i] = (up ? d[i + n] : d[i]) + got;
    }
  }
#pragma unroll
  for (int o = LPP / kBatch / 2; o > 0; o >>= 1) d[0] += __shfl_xor_sync(0xffffffffu, d[0], o);
  *which = w;
  return d[0];
}

// LPP: lanes a position (8, 16 or 32), 0 for fewer (head sizes below 32).
template <int LPP, int R, int NT>
__global__ void __launch_bounds__(NT) k_pattn_few(const FewParams f) {
  extern __shared__ __align__(16) uint8_t smem[];
  const PAttnParams& p = f.a;
  const uint32_t hd = p.pool.hd, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t C = cluster_size(), rank = cluster_rank();
  const uint32_t seq = blockIdx.x / C, kvh = blockIdx.y, v0 = blockIdx.z * R;
  const Sequence sq = load_sequence(p.batch, seq, p.pool.page_shift);
  if (!sq.ok) {  // (the whole cluster leaves)
    if (tid == 0 && rank == 0) note(p.batch, seq, err_key(0, p.pool.layer, CK_PAGED_BAD_SEQUENCE, 0));
    return;
  }
  const uint32_t group = p.heads / p.pool.kv_heads, queries = sq.count * group;
  if (v0 >= queries) return;
  const uint32_t nv = min((uint32_t)R, queries - v0);
  // positions each query sees: those up to its row's own
  uint32_t np[R], top = 0;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const uint32_t up = (v0 + r) / group + sq.len;  // position + count
    np[r] = r < nv && up >= sq.count ? up - sq.count + 1 : 0;
    top = max(top, np[r]);
  }
  const uint32_t per = (top + C - 1) / C, c0 = min(top, rank * per), n = min(top, c0 + per) - c0;
  const FewLayout w = few_layout<NT, R>(hd, f.ids, f.cap, f.sc_smem);
  int4* vpre = reinterpret_cast<int4*>(smem + w.vpre);
  unsigned long long* part = reinterpret_cast<unsigned long long*>(smem + w.part);
  int64_t* q_s = reinterpret_cast<int64_t*>(smem + w.q);
  unsigned long long* red = reinterpret_cast<unsigned long long*>(smem + w.red);
  unsigned long long* xm = red + (NT / 32) * R;
  unsigned long long* xz = xm + R;
  uint32_t* ids = reinterpret_cast<uint32_t*>(smem + w.ids);
  const size_t block = ((size_t)blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
  long long* sc = f.sc_smem ? reinterpret_cast<long long*>(smem + w.sc) : f.scores + block * R * f.cap;

  const uint32_t shift = p.pool.page_shift, mask = (1u << shift) - 1, page0 = c0 >> shift;
  const uint32_t* table = p.batch.table + (size_t)seq * p.batch.stride;
  for (uint32_t i = tid; n != 0 && i <= ((c0 + n - 1) >> shift) - page0; i += NT) {
    const uint32_t id = table[page0 + i];
    ids[i] = id;
    if (id >= p.pool.pages) note(p.batch, seq, err_key((page0 + i) << shift, p.pool.layer, CK_PAGED_BAD_PAGE, 0));
  }
  int wide = 0;
  for (uint32_t i = tid; i < R * hd; i += NT) {
    const uint32_t r = i / hd, v = v0 + r;
    int64_t x = 0;
    if (r < nv)
      x = p.q[(size_t)(sq.first + v / group) * p.q_stride + (size_t)(kvh * group + v % group) * hd + i % hd];
    q_s[i] = x;
    wide |= x != (int32_t)x;
  }
  wide = __syncthreads_or(wide);

  const uint32_t lpp = LPP ? LPP : hd / 4, ppw = 32 / lpp, sub = lane % lpp, slot = lane / lpp, e0 = 4 * sub;
  const uint32_t step = (NT / 32) * ppw, round = step * kBatch;
  // position c0 + i of the pool, this lane's four words (zeros outside the range or the pool)
  auto at = [&](const int32_t* pool, uint32_t i) -> const int4* {
    if (i >= n) return nullptr;
    const uint32_t t = c0 + i, id = ids[(t >> shift) - page0];
    if (id >= p.pool.pages) return nullptr;
    return reinterpret_cast<const int4*>(pool + page_word(p.pool, id, kvh) + (size_t)(t & mask) * hd + e0);
  };
  // the first values travel while the scores are formed
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    const int4* src = at(p.pool.v, b * step + warp * ppw + slot);
    if (src)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_of(vpre + b * NT + tid)), "l"(src)
                   : "memory");
    else
      vpre[b * NT + tid] = make_int4(0, 0, 0, 0);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");

  // scores
  long long m[R];
#pragma unroll
  for (int r = 0; r < R; ++r) m[r] = LLONG_MIN;
  auto score = [&](int r, uint32_t i, unsigned long long d) {
    if (i >= n) return;
    const long long v = wmul((long long)d >> 16, (int64_t)p.inv_sqrt) >> 24;
    sc[(size_t)r * f.cap + i] = v;
    if (c0 + i < np[r]) m[r] = max(m[r], v);
  };
  for (uint32_t base = 0; base < n; base += round) {
    int4 k4[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int4* src = at(p.pool.k, base + b * step + warp * ppw + slot);
      k4[b] = src ? __ldg(src) : make_int4(0, 0, 0, 0);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t q0 = q_s[r * hd + e0], q1 = q_s[r * hd + e0 + 1], q2 = q_s[r * hd + e0 + 2],
                    q3 = q_s[r * hd + e0 + 3];
      unsigned long long d[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b)  // the low words as signed 32-bit factors
        d[b] = (unsigned long long)((long long)(int32_t)q0 * k4[b].x) +
               (unsigned long long)((long long)(int32_t)q1 * k4[b].y) +
               (unsigned long long)((long long)(int32_t)q2 * k4[b].z) +
               (unsigned long long)((long long)(int32_t)q3 * k4[b].w);
      if (wide) {  // and what is left of the queries above them, times 2^32
        const uint32_t h0 = (uint32_t)((q0 - (int32_t)q0) >> 32), h1 = (uint32_t)((q1 - (int32_t)q1) >> 32),
                       h2 = (uint32_t)((q2 - (int32_t)q2) >> 32), h3 = (uint32_t)((q3 - (int32_t)q3) >> 32);
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
          d[b] += (unsigned long long)(h0 * (uint32_t)k4[b].x + h1 * (uint32_t)k4[b].y + h2 * (uint32_t)k4[b].z +
                                       h3 * (uint32_t)k4[b].w)
                  << 32;
      }
      if constexpr (LPP >= kBatch) {
        uint32_t b;
        const unsigned long long s = group_sums<LPP>(d, sub, &b);
        if (sub % (LPP / kBatch) == 0) score(r, base + b * step + warp * ppw + slot, s);
      } else {
        for (uint32_t o = lpp >> 1; o > 0; o >>= 1) {
#pragma unroll
          for (int b = 0; b < kBatch; ++b) d[b] += __shfl_xor_sync(0xffffffffu, d[b], o);
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
          if (sub == 0) score(r, base + b * step + warp * ppw + slot, d[b]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m[r] = max(m[r], __shfl_xor_sync(0xffffffffu, m[r], o));
    if (lane == 0) red[warp * R + r] = (unsigned long long)m[r];
  }
  __syncthreads();
  if (tid < R) {
    long long v = LLONG_MIN;
    for (int k = 0; k < (NT / 32); ++k) v = max(v, (long long)red[k * R + tid]);
    xm[tid] = (unsigned long long)v;
  }
  if (C > 1) cluster_sync();
  else __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = (long long)xm[r];
    if (C > 1) {  // lane k asks block k
      if (lane < C) m[r] = (long long)peer_word(xm + r, lane);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) m[r] = max(m[r], __shfl_xor_sync(0xffffffffu, m[r], o));
      m[r] = __shfl_sync(0xffffffffu, m[r], 0);
    }
  }
  // exponentials and their sums
  unsigned long long z[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    z[r] = 0;
    const uint32_t seen = np[r] > c0 ? min(n, np[r] - c0) : 0;
    long long* s = sc + (size_t)r * f.cap;
    for (uint32_t i = tid; i < n; i += NT) {
      const uint32_t e = i < seen ? exponential(p.exp_tab, (unsigned long long)m[r] - (unsigned long long)s[i]) : 0;
      s[i] = e;
      z[r] += e;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z[r] += __shfl_xor_sync(0xffffffffu, z[r], o);
    if (lane == 0) red[warp * R + r] = z[r];
  }
  __syncthreads();
  if (tid < R) {
    unsigned long long v = 0;
    for (int k = 0; k < (NT / 32); ++k) v += red[k * R + tid];
    xz[tid] = v;
  }
  if (C > 1) cluster_sync();
  else __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    z[r] = xz[r];
    if (C > 1) {
      z[r] = lane < C ? peer_word(xz + r, lane) : 0;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) z[r] += __shfl_xor_sync(0xffffffffu, z[r], o);
      z[r] = __shfl_sync(0xffffffffu, z[r], 0);
    }
    if (z[r] < kOne) z[r] = kOne;
    const float rz = rcp_estimate((float)z[r]);
    long long* s = sc + (size_t)r * f.cap;
    for (uint32_t i = tid; i < n; i += NT)
      s[i] = (long long)div_by_estimate((unsigned long long)s[i] << 24, z[r], rz);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  // weighted values
  unsigned long long a[R][4];
#pragma unroll
  for (int r = 0; r < R; ++r) a[r][0] = a[r][1] = a[r][2] = a[r][3] = 0;
  for (uint32_t base = 0; base < n; base += round) {
    int4 v4[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (base == 0) {
        v4[b] = vpre[b * NT + tid];
      } else {
        const int4* src = at(p.pool.v, base + b * step + warp * ppw + slot);
        v4[b] = src ? __ldg(src) : make_int4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const uint32_t i = base + b * step + warp * ppw + slot;
        const long long pb = i < n ? (int32_t)sc[(size_t)r * f.cap + i] : 0;  // P <= 2^24
        a[r][0] += (unsigned long long)(pb * v4[b].x);
        a[r][1] += (unsigned long long)(pb * v4[b].y);
        a[r][2] += (unsigned long long)(pb * v4[b].z);
        a[r][3] += (unsigned long long)(pb * v4[b].w);
      }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    for (uint32_t o = 16; o >= lpp; o >>= 1) {
#pragma unroll
      for (int j = 0; j < 4; ++j) a[r][j] += __shfl_xor_sync(0xffffffffu, a[r][j], o);
    }
    if (slot == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) part[((size_t)warp * R + r) * hd + e0 + j] = a[r][j];
    }
  }
  __syncthreads();
  for (uint32_t i = tid; i < R * hd; i += NT) {
    unsigned long long t = 0;
    for (int k = 0; k < (NT / 32); ++k) t += part[(size_t)k * R * hd + i];
    part[i] = t;  // (only this thread reads or writes entry i of any warp)
  }
  if (C > 1) cluster_sync();
  // a slice of the outputs each block
  for (uint32_t i = rank * NT + tid; i < nv * hd; i += C * NT) {
    unsigned long long t = 0;
    if (C > 1) {
      unsigned long long w[8];
#pragma unroll
      for (uint32_t k = 0; k < 8; ++k) w[k] = k < C ? peer_word(part + i, k) : 0;
#pragma unroll
      for (uint32_t k = 0; k < 8; ++k) t += w[k];
    } else {
      t = part[i];
    }
    const uint32_t v = v0 + i / hd;
    p.out[((size_t)(sq.first + v / group) * p.heads + kvh * group + v % group) * hd + i % hd] = (long long)t >> 24;
  }
  if (C > 1) cluster_sync();  // no block leaves while another reads its sums
}

struct FewPlan {
  bool use;
  uint32_t NT, R, C, z, cap, ids;
  bool sc_smem;
  uint32_t smem;
  uint64_t work;
};

template <int NT>
uint32_t few_smem(uint32_t R, uint32_t hd, uint32_t ids, uint32_t cap, bool sc_smem) {
  return R == 1   ? few_layout<NT, 1>(hd, ids, cap, sc_smem).size
         : R == 2 ? few_layout<NT, 2>(hd, ids, cap, sc_smem).size
                  : few_layout<NT, 4>(hd, ids, cap, sc_smem).size;
}

FewPlan plan_few(const ck_paged_cache& c, const ck_paged_batch& b, uint32_t heads, const DeviceFacts& f) {
  FewPlan w = {};
  const uint64_t queries = (uint64_t)b.max_new * (heads / c.kv_heads);
  w.R = queries == 1 ? 1 : queries == 2 ? 2 : 4;
  w.z = (uint32_t)((queries + w.R - 1) / w.R);
  // blocks of a cluster: until two an SM are there, while each has 256 positions
  const uint64_t items = (uint64_t)b.seqs * c.kv_heads * w.z;
  w.C = 1;
  while (w.C < 8 && items * w.C < 2ull * f.sms && b.max_len / (2 * w.C) >= 256) w.C *= 2;
  w.NT = items * w.C >= 4ull * f.sms ? kNarrow : 256;
  w.cap = (b.max_len + w.C - 1) / w.C;
  w.ids = w.cap / c.page + 2;
  auto smem = [&](bool sc) {
    return w.NT == 256 ? few_smem<256>(w.R, c.head_dim, w.ids, w.cap, sc)
                       : few_smem<kNarrow>(w.R, c.head_dim, w.ids, w.cap, sc);
  };
  w.sc_smem = smem(true) <= (uint32_t)f.optin / 2 - 2048;
  w.smem = smem(w.sc_smem);
  w.work = w.sc_smem ? 0 : 8ull * w.cap * w.R * items * w.C;
  w.use = w.smem <= (uint32_t)f.optin && w.z <= 65535;
  return w;
}

template <int LPP, int R, int NT>
cudaError_t launch_few(const FewParams& p, const FewPlan& w, const DeviceFacts& f, cudaStream_t s) {
  static std::atomic<bool> ready[64];
  if (!ready[f.dev].load(std::memory_order_relaxed)) {
    const cudaError_t e =
        cudaFuncSetAttribute(k_pattn_few<LPP, R, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, f.optin);
    if (e != cudaSuccess) return e;
    ready[f.dev].store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.a.batch.seqs * w.C, p.a.pool.kv_heads, w.z);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = w.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = w.C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_pattn_few<LPP, R, NT>, p);
}

template <int R, int NT>
cudaError_t launch_few_lpp(const FewParams& p, const FewPlan& w, const DeviceFacts& f, cudaStream_t s) {
  switch (p.a.pool.hd) {
    case 128: return launch_few<32, R, NT>(p, w, f, s);
    case 64: return launch_few<16, R, NT>(p, w, f, s);
    case 32: return launch_few<8, R, NT>(p, w, f, s);
    default: return launch_few<0, R, NT>(p, w, f, s);
  }
}

template <int NT>
cudaError_t launch_few_r(const FewParams& p, const FewPlan& w, const DeviceFacts& f, cudaStream_t s) {
  return w.R == 1   ? launch_few_lpp<1, NT>(p, w, f, s)
         : w.R == 2 ? launch_few_lpp<2, NT>(p, w, f, s)
                    : launch_few_lpp<4, NT>(p, w, f, s);
}

// Which kernel a call takes, by the queries a key head has at most (rows x heads that share it):
// a few go to k_pattn_few, more of head size 64 or 128 to the tensor cores, with k_pattn_rows
// behind them for tiles with values beyond their digits; small heads in any number to
// k_pattn_few as long as its grid holds them.
struct AttentionPlan {
  FewPlan few;
  TilesPlan tiles;
  uint32_t rows_blocks;
  uint64_t work;
};
AttentionPlan attention_plan(const ck_paged_cache& c, const ck_paged_batch& b, uint32_t heads, const DeviceFacts& f) {
  AttentionPlan w = {};
  const uint64_t queries = (uint64_t)b.max_new * (heads / c.kv_heads);
  if (queries > kFewQueries) w.tiles = plan_tiles(c, b, heads, f);
  if (!w.tiles.use) w.few = plan_few(c, b, heads, f);
  if (w.few.use) {
    w.work = std::max<uint64_t>(align256(w.few.work), 256);  // never an empty buffer
    return w;
  }
  // four blocks an SM are resident; no more than there are items or places for their scores
  const uint64_t items = (uint64_t)b.rows * heads, line = 8ull * b.max_len;
  w.rows_blocks = (uint32_t)std::min<uint64_t>(items, 4ull * f.sms);
  if (w.tiles.use) {
    w.rows_blocks = (uint32_t)std::min<uint64_t>(w.rows_blocks, (w.tiles.sums_off - w.tiles.scores_off) / line);
    w.work = align256(w.tiles.size);
  } else {
    w.work = align256(w.rows_blocks * line);
  }
  return w;
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
  *out = attention_plan(*cache, *batch, heads, f).work;
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
  DeviceFacts f;
  CKP_CUDA(device_facts(&f));
  const AttentionPlan plan = attention_plan(*cache, *batch, heads, f);
  if (work_len < plan.work) return CK_BUFFER_TOO_SMALL;
  const PAttnParams p = {pool_view(*cache, layer), batch_view(*batch), dev_q, q_stride, heads, inv_sqrt, dev_exp, dev_out};
  uint8_t* work = static_cast<uint8_t*>(dev_work);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (plan.few.use) {
    const FewParams fp = {p, reinterpret_cast<long long*>(work), plan.few.cap, plan.few.ids, plan.few.sc_smem};
    CKP_CUDA(plan.few.NT == 256 ? launch_few_r<256>(fp, plan.few, f, s) : launch_few_r<kNarrow>(fp, plan.few, f, s));
    return CK_OK;
  }
  RowsParams rp = {p, reinterpret_cast<long long*>(work), nullptr, nullptr, 0};
  if (plan.tiles.use) {
    CKP_CUDA(cudaMemsetAsync(work + plan.tiles.any_off, 0, 4, s));
    const TilesParams tp = {p, plan.tiles.tiles, plan.tiles.cap, reinterpret_cast<uint32_t*>(work + plan.tiles.any_off),
                            reinterpret_cast<uint32_t*>(work + plan.tiles.away_off),
                            reinterpret_cast<int32_t*>(work + plan.tiles.scores_off),
                            reinterpret_cast<ulonglong2*>(work + plan.tiles.sums_off)};
    CKP_CUDA(launch_tiles(tp, plan.tiles, f, s));
    rp.scores = reinterpret_cast<long long*>(work + plan.tiles.scores_off);
    rp.any = tp.any;
    rp.away = tp.away;
    rp.tiles = plan.tiles.tiles;
  }
  k_pattn_rows<<<plan.rows_blocks, kRowsThreads, 0, s>>>(rp);
  CKP_CUDA(cudaGetLastError());
  return CK_OK;
}

}  // extern "C"
