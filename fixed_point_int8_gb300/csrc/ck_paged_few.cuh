// Attention of a few new tokens over a cache in pages ("Attention, stage by stage"): the kernel,
// its plan and its launch, for the whole cache and for a window of it (each compiled by itself).
#pragma once
#include "ck_paged_attention.cuh"

namespace ck {

// ------------------------------------------------------------------ a few queries a key head

// A cluster of blocks takes up to R queries (rows x heads that share a key head) of one sequence
// and one key head, each block a range of positions, so that every key and value word is read
// once: scores into the block's scratch, maximum and sum exchanged through distributed shared
// memory, weighted values summed over the cluster.  HBM bounds it once the positions are many;
// below, the instructions around the exchanges.  LPP lanes take a position, NCH chunks of four
// elements each (eight lanes and two chunks for head size 64: adding up over few lanes is what
// the scores cost: a block of 128 positions takes 11,700 warp instructions with sixteen lanes,
// 6,000 with eight).  Keys and then values stream through a ring of asynchronous copies, kBatch positions a
// lane group each; a lane copies the words that it uses itself, so nothing waits on another
// lane, and the values are on their way while the exponentials are formed.  One token over 8,191
// positions of 32 heads: 134 MB in 28.9 us (4.6 TB/s); 64 runs of 65 to 191: 30.1 us, 20 of them
// without any load.
// With a window the places that any of the queries sees follow one another (Span), and the others
// are neither read nor counted; of those, each query takes what it sees itself.  One token with the last
// 2,048 of 8,191 positions and the first four, 32 heads: 34 MB in 14.4 us (in clusters of four with twice
// the threads 16.4); 64 streams with 1,024 and four: 1.08 GB in 172 us (6.3 TB/s, 92 % of the copy rate).
constexpr uint32_t kMaxCluster = 16;
constexpr int kNarrow = 64, kMiddle = 128, kBroad = 256;  // threads of a block
constexpr unsigned long long kNowhere = ~0ull;

struct FewParams {
  PAttnParams a;
  long long* scores;     // [blocks][R][cap], where they do not fit shared memory
  uint32_t cap;          // positions a block takes at most
  uint32_t ids;          // table entries a block holds
  uint32_t sc_smem;      // the scores lie in shared memory
  uint32_t split;        // log2 of the cluster's blocks
  uint32_t seq0, z0;     // first sequence and first group of R queries of this launch
};

// Scores that do not fit shared memory take R * cap words of the scratch a block; those of every group
// of queries at once would be gigabytes (4 GB for a chunk of 2,048 rows over 8,192 positions of 32 key
// heads of 32).  Past kFewScratch, launches that follow one another share it, each of whole sequences
// or, of one sequence, of some groups of queries.  Each ends with SMs idle: that chunk takes 11.8 ms in
// two launches, 11.6 in one and 13.0 in eight of 512 MB; fewer blocks that loop took 16.6.
constexpr uint64_t kFewScratch = 2ull << 30;
constexpr uint64_t kFewLaunches = 64;
struct FewPlan {
  bool use;
  uint32_t NT, R, C, z, cap, ids;
  uint32_t seqs_each, z_each;  // sequences and groups of queries of one launch
  bool sc_smem;
  uint32_t smem;
  uint64_t work;
};

// The launches of a plan, for the whole cache and for windows of it.
cudaError_t launch_few_whole(const FewParams& p, const FewPlan& w, const DeviceFacts& f, cudaStream_t s);
cudaError_t launch_few_window(const FewParams& p, const FewPlan& w, const DeviceFacts& f, cudaStream_t s);

namespace {

__device__ __forceinline__ uint32_t smem_of(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
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

// Batches in flight and the one at work.
// Positions a lane group takes at once: fewer where four queries' sums fill the registers, and
// where many small blocks share an SM.
__host__ __device__ constexpr int few_batch(int nt, int r) { return r == 4 || nt == kNarrow ? 4 : 8; }
__host__ __device__ constexpr int few_stages(int nt, int nch) { return nt == kBroad ? 4 - nch : 5 - nch; }
struct FewLayout {
  uint32_t ring, part, q, red, ids, sc, size;
};
template <int NT, int R>
__host__ __device__ inline FewLayout few_layout(int nch, uint32_t hd, uint32_t ids, uint32_t cap, bool sc_smem) {
  FewLayout w;
  uint32_t off = 0;
  w.ring = off; off += few_stages(NT, nch) * nch * few_batch(NT, R) * NT * 16;
  w.part = off; off += (NT / 32) * R * hd * 8;
  w.q = off; off += R * hd * 8;
  w.red = off; off += (2 * (NT / 32) + 2) * R * 8;
  w.ids = off; off += (ids * 8 + 15) & ~15u;
  w.sc = off; off += sc_smem ? R * cap * 8 : 0;
  w.size = off;
  return w;
}

// Sums d[0 .. N) over the LPP lanes of a group; lane `sub` ends with the sum of batch entry
// *which.  The first steps halve what a lane carries, so that 8 sums cost 7 exchanges.
template <int LPP, int N>
__device__ __forceinline__ unsigned long long group_sums(unsigned long long (&d)[N], uint32_t sub,
                                                         uint32_t* which) {
  uint32_t w = 0;
#pragma unroll
  for (int n = N / 2, o = LPP / 2; n > 0; n >>= 1, o >>= 1) {
    const bool up = sub & o;
    w = 2 * w + up;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const unsigned long long got = __shfl_xor_sync(0xffffffffu, up ? d[i] : d[i + n], o);
      d[i] = (up ? d[i + n] : d[i]) + got;
    }
  }
#pragma unroll
  for (int o = LPP / N / 2; o > 0; o >>= 1) d[0] += __shfl_xor_sync(0xffffffffu, d[0], o);
  *which = w;
  return d[0];
}

// The largest of the warp's values, and the sum of its values below 2^55, by 32-bit reductions.
__device__ __forceinline__ long long warp_max(long long v) {
  const int32_t hi = __reduce_max_sync(0xffffffffu, (int32_t)(v >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (int32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return (long long)((unsigned long long)(uint32_t)hi << 32 | lo);
}
__device__ __forceinline__ unsigned long long warp_total(unsigned long long v) {
  const uint32_t lo = __reduce_add_sync(0xffffffffu, (uint32_t)v & 0x7FFFFFFu);  // 27 bits of each
  const uint32_t hi = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 27));
  return ((unsigned long long)hi << 27) + lo;
}

// LPP = 0: hd / 4 lanes a position (head sizes below 32).
template <int LPP, int NCH, int R, int NT, bool WINDOW>
__global__ void __launch_bounds__(NT) k_pattn_few(const FewParams f) {
  constexpr int kStages = few_stages(NT, NCH), kBatch = few_batch(NT, R), kWarps = NT / 32;
  extern __shared__ __align__(16) uint8_t smem[];
  const PAttnParams& p = f.a;
  const uint32_t hd = LPP ? 4 * LPP * NCH : p.pool.hd;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t C = 1u << f.split, rank = blockIdx.x & (C - 1);
  const uint32_t seq = f.seq0 + (blockIdx.x >> f.split), kvh = blockIdx.y, v0 = (f.z0 + blockIdx.z) * R;
  const Sequence sq = load_sequence(p.batch, seq, p.pool.page_shift);
  if (!sq.ok) {  // (the whole cluster leaves)
    if (tid == 0 && rank == 0) note(p.batch, seq, err_key(0, p.pool.layer, CK_PAGED_BAD_SEQUENCE, 0));
    return;
  }
  const uint32_t group = p.heads / p.pool.kv_heads, queries = sq.count * group;
  if (v0 >= queries) return;
  // each query's row and head, and the positions it sees: those up to its row's own
  uint32_t np[R], row[R], head[R], top = 0, pos0 = 0xFFFFFFFFu;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const uint32_t token = group == 1 ? v0 + r : (v0 + r) / group, up = token + sq.len;  // position + count
    const bool live = v0 + r < queries;
    np[r] = live && up >= sq.count ? up - sq.count + 1 : 0;
    row[r] = sq.first + token;
    head[r] = kvh * group + (v0 + r - token * group);
    top = max(top, np[r]);
    if (WINDOW && np[r]) pos0 = min(pos0, np[r] - 1);
  }
  // with a window: from here on places, of which query r sees those below np[r] that are below
  // `sinks` or not below from[r]
  Span span = {0, 0};
  uint32_t from[R];
  if (WINDOW && top) {
    span = window_span(p, pos0);
    top -= span.skip;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      from[r] = np[r] ? window_begin(p, np[r] - 1) - span.skip : 0;
      np[r] = np[r] ? np[r] - span.skip : 0;
    }
  }
  auto sees = [&](int r, uint32_t u) { return u < np[r] && (!WINDOW || u < p.sinks || u >= from[r]); };
  const uint32_t per = (top + C - 1) >> f.split, c0 = min(top, rank * per), n = min(top, c0 + per) - c0;
  const FewLayout w = few_layout<NT, R>(NCH, hd, f.ids, f.cap, f.sc_smem);
  int4* ring = reinterpret_cast<int4*>(smem + w.ring);
  unsigned long long* part = reinterpret_cast<unsigned long long*>(smem + w.part);
  int64_t* q_s = reinterpret_cast<int64_t*>(smem + w.q);
  unsigned long long* redm = reinterpret_cast<unsigned long long*>(smem + w.red);  // [warp][R]
  unsigned long long* redz = redm + kWarps * R;
  unsigned long long* xm = redz + kWarps * R;
  unsigned long long* xz = xm + R;
  unsigned long long* pages = reinterpret_cast<unsigned long long*>(smem + w.ids);  // first bytes of the block's pages
  const size_t block = ((size_t)blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
  long long* sc = f.sc_smem ? reinterpret_cast<long long*>(smem + w.sc) : f.scores + block * R * f.cap;

  const uint32_t shift = p.pool.page_shift, mask = (1u << shift) - 1, page0 = c0 >> shift;
  const uint32_t* table = p.batch.table + (size_t)seq * p.batch.stride;
  // The block's pages: those of its places below the span's edge, and from `second` on in the list those of
  // the others, the first of which is page1.
  uint32_t listed = n != 0 ? ((c0 + n - 1) >> shift) - page0 + 1 : 0, second = 0, page1 = 0;
  if (WINDOW && n != 0) {
    second = c0 < span.edge ? ((min(c0 + n, span.edge) - 1) >> shift) - page0 + 1 : 0;
    page1 = (max(c0, span.edge) + span.skip) >> shift;
    listed = second + (c0 + n > span.edge ? ((c0 + n - 1 + span.skip) >> shift) - page1 + 1 : 0);
  }
  int holes = 0;  // a page outside the pool
  for (uint32_t i = tid; i < listed; i += NT) {
    const uint32_t at = !WINDOW || i < second ? page0 + i : page1 + i - second, id = table[at];
    pages[i] = id < p.pool.pages ? 4 * page_word(p.pool, id, kvh) : kNowhere;
    if (id >= p.pool.pages) {
      note(p.batch, seq, err_key(at << shift, p.pool.layer, CK_PAGED_BAD_PAGE, 0));
      holes = 1;
    }
  }
  int wide = 0;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t* q = p.q + row[r] * p.q_stride + head[r] * hd;
    for (uint32_t i = tid; i < hd; i += NT) {
      const int64_t x = v0 + r < queries ? q[i] : 0;
      q_s[r * hd + i] = x;
      wide |= x != (int32_t)x;
    }
  }
  wide = __syncthreads_or(wide);
  holes = __syncthreads_or(holes);

  const uint32_t lpp = LPP ? LPP : hd / 4, ppw = 32 / lpp, sub = lane % lpp, slot = lane / lpp, e0 = 4 * sub;
  const uint32_t step = kWarps * ppw, round = step * kBatch;  // chunk c of a lane: elements e0 + 4 c lpp ..
  // Batch g of the stream: keys of round g, then values of round g - rounds.  This lane's words of
  // its kBatch positions go to its places of slot g % kStages: zeros of a page outside the pool,
  // and those of the last position again behind it.
  const uint32_t rounds = (n + round - 1) / round;
  uint32_t sent = 0;
  auto send = [&] {
    if (sent < 2 * rounds) {
      const bool keys = sent < rounds;
      const char* pool = reinterpret_cast<const char*>((keys ? p.pool.k : p.pool.v) + e0);
      const uint32_t first = (keys ? sent : sent - rounds) * round + warp * ppw + slot;
      const uint32_t to = smem_of(ring + (sent % kStages) * NCH * kBatch * NT + tid);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        uint32_t u = (c0 & mask) + min(first + b * step, n - 1);  // from the first page's start
        if (WINDOW) {  // (and here a page of the list and a place in it)
          const uint32_t place = c0 + min(first + b * step, n - 1);
          u = place < span.edge ? place - (page0 << shift) : place + span.skip - ((page1 - second) << shift);
        }
        unsigned long long at = pages[u >> shift];
        uint32_t bytes = 16;
        if (holes && at == kNowhere) at = bytes = 0;
        const char* src = pool + (at + (u & mask) * (4 * hd));
#pragma unroll
        for (int c = 0; c < NCH; ++c)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + (c * kBatch + b) * NT * 16),
                       "l"(src + 16 * c * lpp), "r"(bytes)
                       : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ++sent;
  };
  uint32_t taken = 0;
  auto take = [&]() -> const int4* {  // the next batch, arrived
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    return ring + (taken++ % kStages) * NCH * kBatch * NT + tid;
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) send();

  // scores
  long long m[R];
#pragma unroll
  for (int r = 0; r < R; ++r) m[r] = LLONG_MIN;
  auto score = [&](int r, uint32_t i, unsigned long long d) {
    if (i >= n) return;
    const long long v = wmul((long long)d >> 16, (int64_t)p.inv_sqrt) >> 24;
    sc[(size_t)r * f.cap + i] = v;
    if (sees(r, c0 + i)) m[r] = max(m[r], v);
  };
  for (uint32_t base = 0; base < n; base += round) {
    const int4* place = take();
    send();  // (into the slot of the batch before, which this lane has used)
    unsigned long long d[R][kBatch];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int b = 0; b < kBatch; ++b) d[r][b] = 0;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      int32_t q[R][4];  // the low words as signed 32-bit factors
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) q[r][j] = (int32_t)q_s[r * hd + e0 + 4 * c * lpp + j];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int4 k4 = place[(c * kBatch + b) * NT];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          d[r][b] += (unsigned long long)((long long)q[r][0] * k4.x);
          d[r][b] += (unsigned long long)((long long)q[r][1] * k4.y);
          d[r][b] += (unsigned long long)((long long)q[r][2] * k4.z);
          d[r][b] += (unsigned long long)((long long)q[r][3] * k4.w);
        }
      }
    }
    if (wide) {  // and what is left of the queries above them, times 2^32
#pragma unroll 1
      for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int64_t* q = q_s + r * hd + e0 + 4 * c * lpp;
          const uint32_t h0 = (uint32_t)((q[0] - (int32_t)q[0]) >> 32), h1 = (uint32_t)((q[1] - (int32_t)q[1]) >> 32),
                         h2 = (uint32_t)((q[2] - (int32_t)q[2]) >> 32), h3 = (uint32_t)((q[3] - (int32_t)q[3]) >> 32);
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            const int4 k4 = place[(c * kBatch + b) * NT];
            d[r][b] += (unsigned long long)(h0 * (uint32_t)k4.x + h1 * (uint32_t)k4.y + h2 * (uint32_t)k4.z +
                                            h3 * (uint32_t)k4.w)
                       << 32;
          }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if constexpr (LPP >= kBatch) {
        uint32_t b;
        const unsigned long long s = group_sums<LPP, kBatch>(d[r], sub, &b);
        if (sub % (LPP / kBatch) == 0) score(r, base + b * step + warp * ppw + slot, s);
      } else {
        for (uint32_t o = lpp >> 1; o > 0; o >>= 1) {
#pragma unroll
          for (int b = 0; b < kBatch; ++b) d[r][b] += __shfl_xor_sync(0xffffffffu, d[r][b], o);
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
          if (sub == 0) score(r, base + b * step + warp * ppw + slot, d[r][b]);
      }
    }
  }
  // the maximum over the block and the cluster
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = warp_max(m[r]);
    if (lane == 0) redm[warp * R + r] = (unsigned long long)m[r];
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int k = 0; k < kWarps; ++k) m[r] = max(m[r], (long long)redm[k * R + r]);
  if (C > 1) {  // lane k asks block k
    if (tid == 0)
#pragma unroll
      for (int r = 0; r < R; ++r) xm[r] = (unsigned long long)m[r];
    cluster_sync();
#pragma unroll
    for (int r = 0; r < R; ++r) m[r] = warp_max(lane < C ? (long long)peer_word(xm + r, lane) : LLONG_MIN);
  }
  // exponentials and their sums
  unsigned long long z[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    z[r] = 0;
    const uint32_t seen = np[r] > c0 ? min(n, np[r] - c0) : 0;
    long long* s = sc + (size_t)r * f.cap;
    for (uint32_t i = tid; i < n; i += NT) {
      const uint32_t e = (WINDOW ? sees(r, c0 + i) : i < seen) ? exponential(p.exp_tab, (unsigned long long)m[r] - (unsigned long long)s[i]) : 0;
      s[i] = e;
      z[r] += e;
    }
    z[r] = warp_total(z[r]);
    if (lane == 0) redz[warp * R + r] = z[r];
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    z[r] = 0;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) z[r] += redz[k * R + r];
  }
  if (C > 1) {
    if (tid == 0)
#pragma unroll
      for (int r = 0; r < R; ++r) xz[r] = z[r];
    cluster_sync();
#pragma unroll
    for (int r = 0; r < R; ++r) z[r] = warp_total(lane < C ? peer_word(xz + r, lane) : 0);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (z[r] < kOne) z[r] = kOne;
    // floor((e << 24) / z) by the reciprocal floor(2^61 / z): short by less than e / 2^37 <= 2^-7,
    // so wrong only when the estimate's fraction ends that close to the next integer
    const uint32_t rz = (uint32_t)div_by_estimate(1ull << 61, z[r], rcp_estimate((float)z[r]));
    long long* s = sc + (size_t)r * f.cap;
    for (uint32_t i = tid; i < rounds * round; i += NT) {  // (zero behind the last position)
      const uint32_t e = i < n ? (uint32_t)s[i] : 0;
      const unsigned long long x = (unsigned long long)e * rz;
      uint32_t q = (uint32_t)(x >> 37);
      if (((uint32_t)(x >> 30) & 0x7Fu) == 0x7Fu) q += ((unsigned long long)e << 24) - (unsigned long long)q * z[r] >= z[r];
      s[i] = q;
    }
  }
  __syncthreads();
  // weighted values
  unsigned long long a[R][NCH][4];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < NCH; ++c) a[r][c][0] = a[r][c][1] = a[r][c][2] = a[r][c][3] = 0;
  for (uint32_t base = 0; base < n; base += round) {
    const int4* place = take();
    send();
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      int4 v4[NCH];
#pragma unroll
      for (int c = 0; c < NCH; ++c) v4[c] = place[(c * kBatch + b) * NT];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        // P <= 2^24: the low word
        const long long pb = reinterpret_cast<const int32_t*>(sc + (size_t)r * f.cap + base + b * step + warp * ppw + slot)[0];
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          a[r][c][0] += (unsigned long long)(pb * v4[c].x);
          a[r][c][1] += (unsigned long long)(pb * v4[c].y);
          a[r][c][2] += (unsigned long long)(pb * v4[c].z);
          a[r][c][3] += (unsigned long long)(pb * v4[c].w);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      for (uint32_t o = 16; o >= lpp; o >>= 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j) a[r][c][j] += __shfl_xor_sync(0xffffffffu, a[r][c][j], o);
      }
      if (slot == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) part[((size_t)warp * R + r) * hd + e0 + 4 * c * lpp + j] = a[r][c][j];
      }
    }
  __syncthreads();
  if (C == 1) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      for (uint32_t i = tid; v0 + r < queries && i < hd; i += NT) {
        unsigned long long t = 0;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) t += part[((size_t)k * R + r) * hd + i];
        p.out[((size_t)row[r] * p.heads + head[r]) * hd + i] = (long long)t >> 24;
      }
    return;
  }
  for (uint32_t i = tid; i < R * hd; i += NT) {
    unsigned long long t = 0;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) t += part[(size_t)k * R * hd + i];
    part[i] = t;  // (only this thread reads or writes entry i of any warp)
  }
  cluster_sync();
  // a slice of the outputs each block
#pragma unroll
  for (int r = 0; r < R; ++r)
    for (uint32_t i = rank * NT + tid; v0 + r < queries && i < hd; i += C * NT) {
      unsigned long long t = 0, word[kMaxCluster];
#pragma unroll
      for (uint32_t k = 0; k < kMaxCluster; ++k) word[k] = k < C ? peer_word(part + r * hd + i, k) : 0;
#pragma unroll
      for (uint32_t k = 0; k < kMaxCluster; ++k) t += word[k];
      p.out[((size_t)row[r] * p.heads + head[r]) * hd + i] = (long long)t >> 24;
    }
  cluster_sync();  // no block leaves while another reads its sums
}

template <int NT>
uint32_t few_smem(uint32_t R, uint32_t hd, uint32_t ids, uint32_t cap, bool sc_smem) {
  const int nch = hd >= 64 ? 2 : 1;
  return R == 1   ? few_layout<NT, 1>(nch, hd, ids, cap, sc_smem).size
         : R == 2 ? few_layout<NT, 2>(nch, hd, ids, cap, sc_smem).size
                  : few_layout<NT, 4>(nch, hd, ids, cap, sc_smem).size;
}

FewPlan plan_few(const ck_paged_cache& c, const ck_paged_batch& b, uint32_t heads, const ck_window* window,
                 const DeviceFacts& f) {
  FewPlan w = {};
  const uint64_t queries = (uint64_t)b.max_new * (heads / c.kv_heads);
  w.R = queries == 1 ? 1 : queries == 2 ? 2 : 4;
  w.z = (uint32_t)((queries + w.R - 1) / w.R);
  const uint32_t line = window_places(window, b.max_len, w.R - 1);
  // blocks of a cluster: until there are two an SM (one, for sixteen), while each has 256 positions
  const uint64_t items = (uint64_t)b.seqs * c.kv_heads * w.z;
  w.C = 1;
  while (w.C < 8 && items * w.C < 2ull * f.sms && line / (2 * w.C) >= 256) w.C *= 2;
  if (w.C == 8 && items * w.C < (uint64_t)f.sms && line >= 16 * 256) w.C = kMaxCluster;
  w.NT = items * w.C <= (uint64_t)f.sms ? kBroad : items * w.C >= 8ull * f.sms && line <= 512 ? kNarrow : kMiddle;
  // (whole rounds: what a block's lanes cover at once)
  const uint32_t lanes = c.head_dim == 128 ? 16 : c.head_dim == 64 ? 8 : c.head_dim / 4, round = w.NT / lanes * few_batch(w.NT, w.R);
  w.cap = ((line + w.C - 1) / w.C + round - 1) / round * round;
  w.ids = w.cap / c.page + (whole(window, b.max_len) ? 2 : 4);  // (a window: two runs of pages)
  auto smem = [&](bool sc) {
    return w.NT == kBroad    ? few_smem<kBroad>(w.R, c.head_dim, w.ids, w.cap, sc)
           : w.NT == kMiddle ? few_smem<kMiddle>(w.R, c.head_dim, w.ids, w.cap, sc)
                             : few_smem<kNarrow>(w.R, c.head_dim, w.ids, w.cap, sc);
  };
  w.sc_smem = smem(true) <= (w.NT == kBroad ? (uint32_t)f.optin : (uint32_t)f.optin / 2 - 2048);
  w.smem = smem(w.sc_smem);
  w.seqs_each = b.seqs;
  w.z_each = w.z;
  if (!w.sc_smem) {
    const uint64_t group = 8ull * w.cap * w.R * w.C * c.kv_heads;  // one sequence's R queries of every key head
    const uint64_t groups = std::max<uint64_t>(1, kFewScratch / group);
    w.z_each = (uint32_t)std::min<uint64_t>(w.z, groups);
    w.seqs_each = (uint32_t)std::min<uint64_t>(b.seqs, std::max<uint64_t>(1, groups / w.z));
    w.work = group * w.z_each * w.seqs_each;
  }
  const uint64_t launches = (uint64_t)((b.seqs + w.seqs_each - 1) / w.seqs_each) * ((w.z + w.z_each - 1) / w.z_each);
  w.use = w.smem <= (uint32_t)f.optin && w.z <= 65535 && launches <= kFewLaunches;
  return w;
}

template <bool WINDOW, int LPP, int NCH, int R, int NT>
cudaError_t launch_few(FewParams p, const FewPlan& w, const DeviceFacts& f, cudaStream_t s) {
  static std::atomic<bool> ready[64];
  if (!ready[f.dev].load(std::memory_order_relaxed)) {
    const cudaError_t e =
        cudaFuncSetAttribute(k_pattn_few<LPP, NCH, R, NT, WINDOW>, cudaFuncAttributeMaxDynamicSharedMemorySize, f.optin);
    if (e != cudaSuccess) return e;
    const cudaError_t e16 =  // clusters of sixteen
        cudaFuncSetAttribute(k_pattn_few<LPP, NCH, R, NT, WINDOW>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e16 != cudaSuccess) return e16;
    ready[f.dev].store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = w.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = w.C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  for (p.seq0 = 0; p.seq0 < p.a.batch.seqs; p.seq0 += w.seqs_each)
    for (p.z0 = 0; p.z0 < w.z; p.z0 += w.z_each) {
      cfg.gridDim = dim3(std::min(w.seqs_each, p.a.batch.seqs - p.seq0) * w.C, p.a.pool.kv_heads, std::min(w.z_each, w.z - p.z0));
      const cudaError_t e = cudaLaunchKernelEx(&cfg, k_pattn_few<LPP, NCH, R, NT, WINDOW>, p);
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

template <bool WINDOW, int R, int NT>
cudaError_t launch_few_lpp(const FewParams& p, const FewPlan& w, const DeviceFacts& f, cudaStream_t s) {
  switch (p.a.pool.hd) {
    case 128: return launch_few<WINDOW, 16, 2, R, NT>(p, w, f, s);
    case 64: return launch_few<WINDOW, 8, 2, R, NT>(p, w, f, s);
    case 32: return launch_few<WINDOW, 8, 1, R, NT>(p, w, f, s);
    default: return launch_few<WINDOW, 0, 1, R, NT>(p, w, f, s);
  }
}

template <bool WINDOW, int NT>
cudaError_t launch_few_r(const FewParams& p, const FewPlan& w, const DeviceFacts& f, cudaStream_t s) {
  return w.R == 1   ? launch_few_lpp<WINDOW, 1, NT>(p, w, f, s)
         : w.R == 2 ? launch_few_lpp<WINDOW, 2, NT>(p, w, f, s)
                    : launch_few_lpp<WINDOW, 4, NT>(p, w, f, s);
}

template <bool WINDOW>
cudaError_t launch_few_any(const FewParams& p, const FewPlan& w, const DeviceFacts& f, cudaStream_t s) {
  return w.NT == kBroad    ? launch_few_r<WINDOW, kBroad>(p, w, f, s)
         : w.NT == kMiddle ? launch_few_r<WINDOW, kMiddle>(p, w, f, s)
                           : launch_few_r<WINDOW, kNarrow>(p, w, f, s);
}

}  // namespace
}  // namespace ck
