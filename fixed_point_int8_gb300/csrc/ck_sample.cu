// Sampling of many rows ("Sampling", the sum and draw passes) with a temperature, top-k, nucleus
// and least-probability filters, and given random numbers.
//
// With D the distance to the row's largest logit and i = floor(256 D / temperature) its place in the
// exponential table (4096 from 16 on), every filter keeps a beginning of the order by (D, token), and all
// tokens of a place weigh the same.  So the counts of the 4,097 places give everything but the
// boundary: the sums of top-k's tokens, how many tokens reach the nucleus, and the place at whose
// tokens the kept ones end, of which the nearest are then chosen by (D, token).  The draw walks
// the kept tokens in the order of the vocabulary, by each warp's sums.
#include <cstddef>
#include <type_traits>

#include "ck_paged.cuh"

namespace ck {
namespace {

struct SampleParams {
  const int64_t* logits;
  size_t stride;
  uint32_t rows, vocab;
  const uint32_t* temperature;
  const uint32_t* top_k;  // null: off, as the next two
  const uint32_t* top_p;
  const uint32_t* min_p;
  const uint64_t* random;
  const uint32_t* exp_tab;
  uint32_t* token;
  uint32_t* prob;
  uint32_t* kept;
  uint32_t split;  // log2 of the blocks of a row's cluster
  uint32_t held;   // they hold its words
  uint32_t ahead;  // rows at work at once
};

constexpr int kDrawThreads = 1024, kDrawWarps = kDrawThreads / 32;
constexpr uint32_t kPer = 16, kBatch = 32 * kPer;          // tokens a lane takes at once, and a warp
constexpr uint32_t kHold = 64 * kBatch;                    // words that a block holds
constexpr uint32_t kBins = 4097, kMine = 5;                // places, and those a thread adds up
constexpr uint32_t kRoom = kMine * kDrawThreads;
constexpr uint32_t kList = 256;                            // tokens at the boundary that are ranked by counting
constexpr uint32_t kAsk = 4096;                            // bytes of a row asked for at a time
constexpr uint32_t kMaxSplit = 8;
constexpr uint32_t kOneQ24 = 1u << 24;
constexpr unsigned long long kNoBound = ~0ull;
static_assert(kRoom >= kBins && kRoom % 4 == 0 && kList <= kDrawThreads && kDrawWarps == 32, "a thread's share");

__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ unsigned long long remote_u64(const void* p, uint32_t rank) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(remote(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint4 remote_v4(const void* p, uint32_t rank) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(remote(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ void put_v4(const void* p, uint32_t rank, uint4 v) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};"
               ::"r"(remote(p, rank)), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void put_u64(const void* p, uint32_t rank, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(remote(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void put_u32(const void* p, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote(p, rank)), "r"(v) : "memory");
}
// (remote accesses to a block's own memory are slower than plain ones)
__device__ __forceinline__ uint32_t remote_count(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], 1;" : "=r"(v) : "r"(remote(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ void row_sync(uint32_t S) {  // the threads of the row's blocks
  if (S > 1)
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  else
    __syncthreads();
}
__device__ __forceinline__ long long warp_max(long long v) {
  const int32_t hi = __reduce_max_sync(0xffffffffu, (int32_t)(v >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (int32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return (long long)((unsigned long long)(uint32_t)hi << 32 | lo);
}
__device__ __forceinline__ uint32_t warp_inclusive_scan32(uint32_t v, uint32_t lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t w = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += w;
  }
  return v;
}
// The warp's number, known to be the same for its lanes: where the compiler doesn't know it, every exchange in
// a branch of one warp first collects the lanes (700 cycles a step of a 64-bit scan).
__device__ __forceinline__ uint32_t warp_number() { return __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0); }
// The sum of the warp's values, each at most 2^34, by 32-bit reductions.
__device__ __forceinline__ unsigned long long warp_sum34(unsigned long long v) {
  const uint32_t lo = __reduce_add_sync(0xffffffffu, (uint32_t)v & 0xFFFFFFu);
  const uint32_t hi = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 24));
  return ((unsigned long long)hi << 24) + lo;
}

// The place of a distance, floor(256 d / t) up to 4096, by one product: with T = t << shift >= 512 and
// D = min(d, 16 t) << shift it is (D * factor + add) >> (32 + down).  factor is 2^(40 + down) / T rounded
// up (add 0), which is exact while 16 T times what the rounding adds to factor * T stays below 2^(32 +
// down), or else rounded down (add = factor / 256: a 256th more in D), which is by the same bound: the two
// add up to T, and 8 T^2 <= 2^(32 + down) with down = floor(log2 T) - 8.
struct Places {
  uint32_t far, factor, shift, down;
  unsigned long long add;
};
__host__ __device__ inline Places places_of(uint32_t t) {
  Places s;
  s.far = 16 * t;
  s.shift = t < 512 ? 9 : 0;
  const unsigned long long T = (unsigned long long)t << s.shift;
  s.down = 0;
  while (T >> (s.down + 10)) ++s.down;  // floor(log2 T) - 9 ..
  ++s.down;
  unsigned long long N = 1ull << (40 + s.down), up = (N + T - 1) / T;
  if (up >> 32) {  // (a power of two)
    --s.down;
    N >>= 1;
    up = (N + T - 1) / T;
  }
  s.factor = (uint32_t)up;
  s.add = 0;
  if (16 * T * (up * T - N) >= 1ull << (32 + s.down)) {
    s.factor = (uint32_t)(N / T);
    s.add = s.factor >> 8;
  }
  return s;
}
__host__ __device__ __forceinline__ uint32_t place_of(uint32_t d, const Places& s) {
  const uint32_t D = (d < s.far ? d : s.far) << s.shift;
  return (uint32_t)(((unsigned long long)D * s.factor + s.add) >> 32) >> s.down;
}
// The first distance of a place.
__device__ __forceinline__ unsigned long long first_of(uint32_t place, uint32_t t) {
  return ((unsigned long long)place * t + 255) >> 8;
}

// Buckets of a distance above the tail's begin, in order: those below 64, then 64 a bit length.
__device__ __forceinline__ uint32_t tail_bucket(unsigned long long x) {
  if (x < 64) return (uint32_t)x;
  const uint32_t e = 63 - (uint32_t)__clzll((long long)x);
  return ((e - 5) << 6) + ((uint32_t)(x >> (e - 6)) & 63u);
}
__device__ __forceinline__ unsigned long long tail_first(uint32_t b) {
  if (b < 64) return b;
  const uint32_t e = (b >> 6) + 5;
  return (1ull << e) + ((unsigned long long)(b & 63u) << (e - 6));
}

// A cluster of blocks a row, warps taking batches of 512 tokens in turn.  A block keeps its part of
// the row as 32-bit words in shared memory, so that HBM is read once and L2 not again; only logits that do
// not fit 32 bits, and vocabularies above 262,144, are read in every pass.  A block fills an SM, so many rows
// follow one another in steps that wait (a row of 32,000: loads 10,000 cycles, counts 7,000, sums 4,500, kept
// weights 5,000, draw 2,500), and the next row's logits are asked for meanwhile: 512 rows take 49 us by
// temperature (2.7 TB/s) and 67 with a nucleus and a least probability, 64 rows 18 on the device, one 13.  Rows
// with masked logits read theirs twice, and those past 32 bits in every pass: 512 take 74 and 89 by temperature.
// Two rows an SM, with 16-bit places in shared memory and the logits read twice, took 55 and 69 us (304 rows in
// flight leave L2), two half rows an SM 48 and 72.  Atomics on shared memory bound the counts, a gather from the
// table the weights.
struct Shared {
  uint32_t hist[kRoom];   // this block's counts, then the row's
  uint32_t table[kRoom];  // the exponentials
  unsigned long long near_d[kList];
  unsigned long long weights[kMaxSplit * kHold / kBatch];  // that are kept, by batch
  unsigned long long red[kDrawWarps], peak, flag, found[3], random;
  uint32_t near_i[kList], n_near;
  uint32_t red_c[kDrawWarps], red_i[kDrawWarps], least, tokens;
  uint32_t f_count, f_rest, f_place;
  Places places;
  __align__(16) int32_t words[1];  // those held; or the weights by batch, where there are more
};
enum Mode { kNarrow32, kMasked32, kWide64 };  // every logit fits 32 bits; those that are not masked do; or not
constexpr int32_t kMaskedWord = INT32_MIN;    // of kMasked32 (where no other logit is as low)

// What is kept: tokens nearer than `first`, and of those from there to `last` the ones up to (d, token).
struct Bound {
  unsigned long long first, last, d;
  uint32_t token;
};

// Number `n` of this warp's batches, of a cluster of 2^split blocks: its number in the row.
__device__ __forceinline__ uint32_t batch_of(uint32_t n, uint32_t split, uint32_t rank, uint32_t warp) {
  return ((n << split) + rank) * kDrawWarps + warp;
}
// The block that has a batch, and the batch's place among the words that the block holds.
__device__ __forceinline__ uint32_t rank_of(uint32_t b, uint32_t split) { return b / kDrawWarps & ((1u << split) - 1); }
__device__ __forceinline__ uint32_t held_at(uint32_t b, uint32_t split) {
  return ((b / kDrawWarps >> split) * kDrawWarps + b % kDrawWarps) * kBatch;
}

template <int MODE, bool HELD>
__device__ __forceinline__ void sample_row(const SampleParams& p, long long m, uint32_t t, uint32_t top_k,
                                           uint32_t top_p, uint32_t min_p, bool filtered) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sm = *reinterpret_cast<Shared*>(smem);
  const uint32_t S = 1u << p.split, rank = blockIdx.x & (S - 1), row = blockIdx.x >> p.split;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = warp_number();
  const long long* l = reinterpret_cast<const long long*>(p.logits) + (size_t)row * p.stride;
  const uint32_t batches = (p.vocab + kBatch - 1) / kBatch;
  using Word = typename std::conditional<MODE == kWide64, long long, int32_t>::type;
  using Distance = typename std::conditional<MODE == kWide64, unsigned long long, uint32_t>::type;
  auto distance = [&](Word x) -> Distance { return (Distance)m - (Distance)x; };
  auto there = [&](Word x) { return MODE == kNarrow32 || (MODE == kMasked32 ? x != (Word)kMaskedWord : (long long)x != LLONG_MIN); };
  const Places places = sm.places;
  auto place = [&](Distance d) {
    return place_of(MODE == kWide64 && (unsigned long long)d >> 31 ? 0x7FFFFFFFu : (uint32_t)d, places);
  };
  // token `at` of batch b
  auto word = [&](uint32_t b, uint32_t at) -> Word {
    if (HELD) return (Word)sm.words[held_at(b, p.split) + at];
    const long long* from = l + b * kBatch + at;
    return MODE == kWide64 ? (Word)__ldg(from) : (Word)__ldg(reinterpret_cast<const int32_t*>(from));
  };
  // Of batch b this lane's tokens that are not masked, `At` words at a time: f(distance, token).  (The loops
  // stay short where they are not the row's work: unrolled throughout, half a megabyte of instructions
  // came through the instruction cache, and the kernel took twice the time.)
  constexpr uint32_t kAtOnce = MODE == kNarrow32 && HELD ? 8 : 4;
  auto each_of = [&](auto at_once, uint32_t b, auto f) {
    constexpr uint32_t At = decltype(at_once)::value;
    const uint32_t i0 = b * kBatch + lane, left = p.vocab - min(p.vocab, i0);
#pragma unroll 1
    for (uint32_t j0 = 0; j0 < kPer; j0 += At) {
      Word x[At];
#pragma unroll
      for (uint32_t j = 0; j < At; ++j) x[j] = HELD || 32 * (j0 + j) < left ? word(b, 32 * (j0 + j) + lane) : 0;
#pragma unroll
      for (uint32_t j = 0; j < At; ++j)
        if (32 * (j0 + j) < left && there(x[j])) f(distance(x[j]), i0 + 32 * (j0 + j));
    }
  };
  // every token of this thread that is not masked
  auto each = [&](auto at_once, auto f) {
#pragma unroll 1
    for (uint32_t n = 0, b; (b = batch_of(n, p.split, rank, warp)) < batches; ++n) each_of(at_once, b, f);
  };
  using Many = std::integral_constant<uint32_t, kAtOnce>;
  using One = std::integral_constant<uint32_t, 1>;

  if (t == 0) {  // the first largest
    uint32_t at = 0xFFFFFFFFu;
    each(Many(), [&](Distance d, uint32_t i) {
      if (d == 0) at = min(at, i);
    });
    at = __reduce_min_sync(0xffffffffu, at);
    if (lane == 0 && at != 0xFFFFFFFFu)
      asm volatile("red.shared::cluster.min.u32 [%0], %1;" ::"r"(remote(&sm.least, 0)), "r"(at) : "memory");
    row_sync(S);
    if (rank == 0 && tid == 0) {
      p.token[row] = sm.least;
      p.prob[row] = kOneQ24;
      p.kept[row] = 1;
    }
    return;
  }

  Bound bound = {kNoBound, kNoBound, kNoBound, 0xFFFFFFFFu};
  uint32_t kept = 0, listed = 0, rest = 0;
  if (filtered) {
    // The row's counts of this thread's buckets, b0 and those behind it, as f names a token's bucket.
    const uint32_t b0 = tid * kMine;
    auto count_all = [&](auto at_once, auto f, uint32_t (&c)[kMine]) {
      uint32_t last = 0;
      each(at_once, [&](Distance d, uint32_t i) {
        const uint32_t b = f(d, i);
        if (b < kBins - 1)
          atomicAdd(sm.hist + b, 1u);
        else
          last += b == kBins - 1;  // (often most of them)
      });
      last = __reduce_add_sync(0xffffffffu, last);
      if (lane == 0 && last) atomicAdd(sm.hist + kBins - 1, last);
      row_sync(S);
      if (S > 1) {
        // each block adds up its share of the places, four a thread, and hands it to all: nobody else touches
        // these words of any block.  (Every thread reading its own places from every block took 10 to 60 us.)
        constexpr uint32_t kQuads = kRoom / 4;
        const uint32_t width = (kQuads + S - 1) / S, q1 = min(kQuads, (rank + 1) * width);
        for (uint32_t q = rank * width + tid; q < q1; q += kDrawThreads) {
          uint4 part[kMaxSplit], sum = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (uint32_t k = 0; k < kMaxSplit; ++k) part[k] = k < S ? remote_v4(sm.hist + 4 * q, k) : sum;
#pragma unroll
          for (uint32_t k = 0; k < kMaxSplit; ++k) {
            sum.x += part[k].x;
            sum.y += part[k].y;
            sum.z += part[k].z;
            sum.w += part[k].w;
          }
          for (uint32_t k = 0; k < S; ++k) put_v4(sm.hist + 4 * q, k, sum);
        }
        row_sync(S);
      }
#pragma unroll
      for (uint32_t j = 0; j < kMine; ++j) c[j] = sm.hist[b0 + j];
    };
    // The bucket in which number `want` (from 1) falls, how many it has, and the number's place in it: of the
    // thread with `before` < want.
    auto find = [&](const uint32_t (&c)[kMine], uint32_t before, uint32_t want) {
#pragma unroll
      for (uint32_t j = 0; j < kMine; ++j) {
        if (before < want && want <= before + c[j]) {
          sm.f_place = b0 + j;
          sm.f_count = c[j];
          sm.f_rest = want - before;
        }
        before += c[j];
      }
    };
    uint32_t c[kMine];
    count_all(Many(), [&](Distance d, uint32_t) { return place(d); }, c);
    // counts and weights before this thread's places
    uint32_t mine = 0, near = 0;
    unsigned long long heavy = 0;
    const unsigned long long least_w = (unsigned long long)min_p * sm.table[0];
#pragma unroll
    for (uint32_t j = 0; j < kMine; ++j) {
      const uint32_t e = sm.table[b0 + j];
      mine += c[j];
      heavy += (unsigned long long)c[j] * e;
      if ((unsigned long long)e << 24 >= least_w) near += c[j];
    }
    const uint32_t count_in = warp_inclusive_scan32(mine, lane);
    const unsigned long long weight_in = warp_inclusive_scan(heavy, lane);
    near = __reduce_add_sync(0xffffffffu, near);
    if (lane == 31) {
      sm.red_c[warp] = count_in;
      sm.red[warp] = weight_in;
      sm.red_i[warp] = near;
    }
    __syncthreads();
    const uint32_t count_to = warp_inclusive_scan32(sm.red_c[lane], lane);
    const unsigned long long weight_to = warp_inclusive_scan(sm.red[lane], lane);
    near = __reduce_add_sync(0xffffffffu, sm.red_i[lane]);
    const uint32_t total = __shfl_sync(0xffffffffu, count_to, 31), ahead_c = __shfl_sync(0xffffffffu, count_to, (warp - 1) & 31u);
    const unsigned long long ahead_w = __shfl_sync(0xffffffffu, weight_to, (warp - 1) & 31u);
    unsigned long long z = __shfl_sync(0xffffffffu, weight_to, 31);
    uint32_t before = count_in - mine + (warp ? ahead_c : 0);
    const unsigned long long weight = weight_in - heavy + (warp ? ahead_w : 0);
    uint32_t keep = top_k ? min(top_k, total) : total;
    if (top_p < kOneQ24) {
      if (keep < total) {  // the weight of the first `keep`
        if (before < keep && keep <= before + mine) {
          uint32_t left = keep - before;
          unsigned long long w = weight;
#pragma unroll
          for (uint32_t j = 0; j < kMine; ++j) {
            const uint32_t take = min(c[j], left);
            w += (unsigned long long)take * sm.table[b0 + j];
            left -= take;
          }
          sm.found[0] = w;
        }
        __syncthreads();
        z = sm.found[0];
      }
      const unsigned long long target = (z >> 24) * top_p + (((z & (kOneQ24 - 1)) * top_p) >> 24);
      if (tid == 0 && target == 0) sm.found[1] = 1;
      if (weight < target && target <= weight + heavy) {
        uint32_t n = before, at = 0;
        unsigned long long w = weight, lack = 0;  // of the place `at`, the first that reaches it
#pragma unroll
        for (uint32_t j = 0; j < kMine; ++j) {
          const unsigned long long here = (unsigned long long)c[j] * sm.table[b0 + j];
          if (w < target && target <= w + here) {
            at = j;
            lack = target - w;
            n = before;
          }
          w += here;
          before += c[j];
        }
        before -= mine;
        const uint32_t e = sm.table[b0 + at];
        n += (uint32_t)((lack + e - 1) / e);
        sm.found[1] = n;
      }
      __syncthreads();
      keep = min(keep, (uint32_t)sm.found[1]);
    }
    if (min_p) keep = max(1u, min(keep, near));
    // the place at which the kept ones end, and how many of it
    if (before < keep && keep <= before + mine) find(c, before, keep);
    __syncthreads();
    kept = keep;
    const uint32_t end = sm.f_place;
    uint32_t among = sm.f_count;
    rest = sm.f_rest;
    unsigned long long lo = first_of(end, t), span = end < 4096 ? first_of(end + 1, t) - lo : 0 - lo;  // (2^64 - lo)
    if (rest == among) {
      bound.first = end < 4096 ? lo + span : kNoBound;
      bound.last = bound.d = end < 4096 ? lo + span - 1 : kNoBound;
    } else if (among <= kList) {
      listed = among;
      bound.first = lo;
      bound.last = lo + (span - 1);
    } else {
      // the nearest `rest` of the `among` at distances lo .. lo + span - 1, by distance and then by token: a step
      // narrows either to one of up to 4,096 buckets
      bool by_token = false, tail = end == 4096;
      uint32_t t_lo = 0, t_span = p.vocab;
      while (rest < among) {
        if (!by_token && span == 1) by_token = true;
        const unsigned long long range = by_token ? t_span : span;
        uint32_t shift = 0;
        while (((range - 1) >> shift) >= 4096) ++shift;
        row_sync(S);  // the counts have been read
        for (uint32_t i = tid; i < kRoom; i += kDrawThreads) sm.hist[i] = 0;
        __syncthreads();
        count_all(One(), [&](Distance d, uint32_t i) {
          const unsigned long long at = by_token ? i - t_lo : d - lo;
          if (d < lo || d - lo >= span || (by_token && (i < t_lo || at >= t_span))) return kBins;
          return tail ? tail_bucket(at) : (uint32_t)(at >> shift);
        }, c);
        mine = 0;
#pragma unroll
        for (uint32_t j = 0; j < kMine; ++j) mine += c[j];
        const uint32_t upto = warp_inclusive_scan32(mine, lane);
        if (lane == 31) sm.red_c[warp] = upto;
        __syncthreads();
        const uint32_t all_to = warp_inclusive_scan32(sm.red_c[lane], lane);
        const uint32_t ahead = __shfl_sync(0xffffffffu, all_to, (warp - 1) & 31u);
        before = upto - mine + (warp ? ahead : 0);
        if (before < rest && rest <= before + mine) find(c, before, rest);
        __syncthreads();
        const uint32_t b = sm.f_place;
        among = sm.f_count;
        rest = sm.f_rest;
        if (by_token) {
          t_lo += b << shift;
          t_span = min(1u << shift, t_span - (b << shift));
        } else {
          const unsigned long long from = tail ? tail_first(b) : (unsigned long long)b << shift;
          const unsigned long long wide = tail ? (b < 64 ? 1ull : 1ull << ((b >> 6) - 1)) : 1ull << shift;
          span = min(wide, span - from);
          lo += from;
          tail = false;
        }
      }
      bound = {lo, lo + (span - 1), lo + (span - 1), by_token ? t_lo + t_span - 1 : 0xFFFFFFFFu};
    }
  }

  // ---- the weights that are kept, by batch, and the tokens at the boundary, to every block
  unsigned long long* weights = HELD ? sm.weights : reinterpret_cast<unsigned long long*>(sm.words);
  const Distance nearest = (Distance)min(bound.first, (unsigned long long)(Distance)~0ull);
  const Distance last = (Distance)min(bound.last, (unsigned long long)(Distance)~0ull);
  auto keeps = [&](Distance d, uint32_t i) {
    return !filtered || d < nearest || (d <= last && (d < bound.d || (d == bound.d && i <= bound.token)));
  };
  uint32_t tokens = 0;
#pragma unroll 1
  for (uint32_t n = 0, b; (b = batch_of(n, p.split, rank, warp)) < batches; ++n) {
    unsigned long long sum = 0;
    bool any = !filtered;
    if (!filtered) {
      each_of(Many(), b, [&](Distance d, uint32_t) {
        sum += sm.table[place(d)];
        if (MODE != kNarrow32) ++tokens;
      });
    } else {
      bool hit = false;
      each_of(Many(), b, [&](Distance d, uint32_t) { hit |= d <= last; });
      any = __any_sync(0xffffffffu, hit);
      if (any) {
        uint32_t border = 0;  // tokens that are ranked first
        each_of(Many(), b, [&](Distance d, uint32_t i) {
          if (d <= last) {
            if (listed ? d < nearest : keeps(d, i))
              sum += sm.table[place(d)];
            else
              border |= 1u << (i / 32 % kPer);
          }
        });
#pragma unroll 1
        for (border = listed ? border : 0; border; border &= border - 1) {
          const uint32_t at = (__ffs((int)border) - 1) * 32 + lane, to = S > 1 ? remote_count(&sm.n_near, 0) : atomicAdd(&sm.n_near, 1u);
          const Distance d = distance(word(b, at));
          if (S == 1) {
            sm.near_d[to] = d;
            sm.near_i[to] = b * kBatch + at;
          }
#pragma unroll 1
          for (uint32_t k = 0; S > 1 && k < S; ++k) {
            put_u64(sm.near_d + to, k, d);
            put_u32(sm.near_i + to, k, b * kBatch + at);
          }
        }
      }
    }
    if (any) {
      __syncwarp();
      sum = warp_sum34(sum);
    }
    if (S == 1 && lane == 0) weights[b] = sum;
    if (S > 1 && lane < S) put_u64(weights + b, lane, sum);
  }
  if (MODE != kNarrow32 && !filtered) {
    tokens = __reduce_add_sync(0xffffffffu, tokens);
    if (lane < S)
      asm volatile("red.shared::cluster.add.u32 [%0], %1;" ::"r"(remote(&sm.tokens, lane)), "r"(tokens) : "memory");
  }
  row_sync(S);
  if (listed) {  // the nearest `rest` of them, by distance and then by token
    if (tid < listed) {
      const unsigned long long d = sm.near_d[tid];
      const uint32_t i = sm.near_i[tid];
      uint32_t r = 0;
      for (uint32_t k = 0; k < listed; ++k) r += sm.near_d[k] < d || (sm.near_d[k] == d && sm.near_i[k] < i);
      if (r < rest) atomicAdd(weights + i / kBatch, (unsigned long long)sm.table[place((Distance)d)]);
      if (r == rest - 1) {
        sm.found[2] = d;
        sm.least = i;
      }
    }
    __syncthreads();
    bound.d = sm.found[2];
    bound.token = sm.least;
  }
  // ---- the draw.  The first warp: the lane whose batches hold it, and the batch.
  if (warp == 0) {
    const uint32_t own = (batches + 31) / 32, g0 = min(batches, lane * own);
    unsigned long long sum = 0;
    for (uint32_t g = 0; g < own; ++g) sum += g0 + g < batches ? weights[g0 + g] : 0;
    const unsigned long long upto = warp_inclusive_scan(sum, lane), z = __shfl_sync(0xffffffffu, upto, 31);
    const unsigned long long draw = z ? sm.random % z : 0;  // (521 cycles; by an estimate of 1 / z 1,120)
    const int holder = z ? __ffs((int)__ballot_sync(0xffffffffu, upto > draw)) - 1 : 0;
    if ((int)lane == holder) {
      unsigned long long rem = draw - (upto - sum);
      uint32_t b = g0;
      while (z && rem >= weights[b]) rem -= weights[b++];
      sm.found[0] = z;
      sm.found[1] = rem;
      sm.f_place = b;
    }
  }
  __syncthreads();
  const unsigned long long z = sm.found[0], rem = sm.found[1];
  const uint32_t b = sm.f_place;
  if (z == 0) {  // (a table of zeros)
    if (rank == 0 && tid == 0) {
      p.token[row] = CK_NO_TOKEN;
      p.prob[row] = 0;
      p.kept[row] = 0;
    }
    return;
  }
  if (rank != rank_of(b, p.split)) return;
  // In the block that has the batch, a thread a token.
  uint32_t e = 0;
  const uint32_t i = b * kBatch + tid;
  if (tid < kBatch && i < p.vocab) {
    const Word x = word(b, tid);
    const Distance d = distance(x);
    if (there(x) && keeps(d, i)) e = sm.table[place(d)];
  }
  const unsigned long long upto = warp_inclusive_scan((unsigned long long)e, lane);
  if (lane == 31) sm.red[warp] = upto;
  __syncthreads();
  if (warp >= kBatch / 32) return;
  unsigned long long ahead = upto - e;
  for (uint32_t w = 0; w < warp; ++w) ahead += sm.red[w];
  if (rem < ahead || rem - ahead >= e) return;
  p.token[row] = i;
  p.prob[row] = (uint32_t)(((unsigned long long)e << 24) / z);
  p.kept[row] = filtered ? kept : MODE != kNarrow32 ? sm.tokens : p.vocab;
}

// (the rare ones by themselves, for the registers of the others)
template <int MODE, bool HELD>
__device__ __noinline__ void sample_row_apart(const SampleParams& p, long long m, uint32_t t, uint32_t top_k,
                                              uint32_t top_p, uint32_t min_p, bool filtered) {
  sample_row<MODE, HELD>(p, m, t, top_k, top_p, min_p, filtered);
}

__global__ void __launch_bounds__(kDrawThreads, 1) k_sample_rows(const __grid_constant__ SampleParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sm = *reinterpret_cast<Shared*>(smem);
  const uint32_t S = 1u << p.split, rank = blockIdx.x & (S - 1), row = blockIdx.x >> p.split;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = warp_number();
  const long long* l = reinterpret_cast<const long long*>(p.logits) + (size_t)row * p.stride;
  const uint32_t batches = (p.vocab + kBatch - 1) / kBatch;
  uint32_t exps[kMine];  // (asked for first, needed after the logits)
#pragma unroll
  for (uint32_t j = 0; j < kMine; ++j) exps[j] = tid + j * kDrawThreads < kBins ? __ldg(p.exp_tab + tid + j * kDrawThreads) : 0;
  const uint32_t t = __ldg(p.temperature + row);
  const uint32_t top_k = p.top_k ? __ldg(p.top_k + row) : 0, top_p = p.top_p ? min(__ldg(p.top_p + row), kOneQ24) : kOneQ24;
  const uint32_t min_p = p.min_p ? min(__ldg(p.min_p + row), kOneQ24) : 0;
  const bool filtered = (top_k != 0 && top_k < p.vocab) || top_p < kOneQ24 || min_p != 0;
  // the row's largest value, and whether any block has a flag
  auto largest = [&](long long v, bool flag, bool* any) {
    v = warp_max(v);
    if (lane == 0) sm.red[warp] = (unsigned long long)v;
    flag = __syncthreads_or(flag);
    v = warp_max((long long)sm.red[lane]);
    if (tid == 0) {
      sm.peak = (unsigned long long)v;
      sm.flag = flag;
    }
    row_sync(S);
    for (uint32_t k = 0; S > 1 && k < S; ++k) {
      v = max(v, (long long)remote_u64(&sm.peak, k));
      flag |= remote_u64(&sm.flag, k) != 0;
    }
    *any = flag;
    return v;
  };
  // ---- the largest logit, of 32 bits, and whether any has more
  int32_t m32 = INT32_MIN, more = 0;
  for (uint32_t n = 0, b; (b = batch_of(n, p.split, rank, warp)) < batches; ++n) {
    const uint32_t i0 = b * kBatch + lane;
    const long long* at = l + i0;
    long long x[kPer];
    if (b * kBatch + kBatch <= p.vocab) {
#pragma unroll
      for (uint32_t j = 0; j < kPer; ++j) x[j] = __ldg(at + 32 * j);
    } else {
#pragma unroll
      for (uint32_t j = 0; j < kPer; ++j) x[j] = i0 + 32 * j < p.vocab ? __ldg(at + 32 * j) : (long long)INT32_MIN;
    }
#pragma unroll
    for (uint32_t j = 0; j < kPer; ++j) {
      if (p.held) sm.words[held_at(b, p.split) + 32 * j + lane] = (int32_t)x[j];
      m32 = max(m32, (int32_t)x[j]);
      more |= (int32_t)(x[j] >> 32) ^ ((int32_t)x[j] >> 31);
    }
  }
#pragma unroll
  for (uint32_t j = 0; j < kMine; ++j) {
    sm.hist[tid + j * kDrawThreads] = 0;
    sm.table[tid + j * kDrawThreads] = min(exps[j], 1u << 30);
  }
  if (tid == 0) {
    sm.n_near = 0;
    sm.tokens = 0;
    sm.least = 0xFFFFFFFFu;
  }
  if (tid == 32) sm.random = __ldg(p.random + row);
  if (tid == 64 && t != 0 && t <= kMaxTemperature) sm.places = places_of(t);
  // The row that a block of this SM takes next, or one near it, comes into L2 while this one is worked on.
  const uint32_t next = row + p.ahead;
  if (warp == 1 && next < p.rows) {
    const uintptr_t from = (reinterpret_cast<uintptr_t>(p.logits + (size_t)next * p.stride) + 15) & ~(uintptr_t)15;
    const uintptr_t to = reinterpret_cast<uintptr_t>(p.logits + (size_t)next * p.stride + p.vocab) & ~(uintptr_t)15;
    for (uintptr_t at = from + (rank * 32 + lane) * (uintptr_t)kAsk; at < to; at += S * 32 * (uintptr_t)kAsk)
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"((uint32_t)min((uintptr_t)kAsk, to - at)) : "memory");
  }
  bool masked = false, wide = false;
  long long m = largest(m32, more != 0, &masked);
  auto none = [&] {
    row_sync(S);  // (every block has read the others' maxima)
    if (rank == 0 && tid == 0) {
      p.token[row] = CK_NO_TOKEN;
      p.prob[row] = 0;
      p.kept[row] = 0;
    }
  };
  if (t > kMaxTemperature) return none();
  if (!masked) {
    if (p.held)
      sample_row<kNarrow32, true>(p, m, t, top_k, top_p, min_p, filtered);
    else
      sample_row_apart<kNarrow32, false>(p, m, t, top_k, top_p, min_p, filtered);
    return;
  }
  // ---- the largest of those that are not masked, and whether any of them has more than 32 bits
  row_sync(S);
  m = LLONG_MIN;
#pragma unroll 1
  for (uint32_t n = 0, b; (b = batch_of(n, p.split, rank, warp)) < batches; ++n)
#pragma unroll 4
    for (uint32_t j = 0; j < kPer; ++j) {
      const uint32_t i = b * kBatch + lane + 32 * j;
      const long long x = i < p.vocab ? __ldg(l + i) : LLONG_MIN;
      m = max(m, x);
      wide |= x != LLONG_MIN && (x != (int32_t)x || x == kMaskedWord);
      if (p.held && x == LLONG_MIN) sm.words[held_at(b, p.split) + 32 * j + lane] = kMaskedWord;
    }
  m = largest(m, wide, &wide);
  if (m == LLONG_MIN) return none();  // every token is masked
  if (p.held && !wide)
    sample_row<kMasked32, true>(p, m, t, top_k, top_p, min_p, filtered);
  else
    sample_row_apart<kWide64, false>(p, m, t, top_k, top_p, min_p, filtered);
}

// Blocks of a row's cluster: as many as hold its words; then more, while there are SMs for them all (a block
// fills one) and every warp has a batch.
uint32_t sample_split(uint32_t rows, uint32_t vocab, const DeviceFacts& f) {
  uint32_t S = 1;
  while (S < kMaxSplit && (S * kHold < vocab || (2ull * S * rows <= (uint64_t)f.sms && S * kDrawWarps * kBatch < vocab))) S *= 2;
  return S;
}

cudaError_t launch_sample(SampleParams p, cudaStream_t s) {
  DeviceFacts f;
  cudaError_t e = device_facts(&f);
  if (e != cudaSuccess) return e;
  static std::atomic<bool> ready[64];
  if (!ready[f.dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(k_sample_rows, cudaFuncAttributeMaxDynamicSharedMemorySize, offsetof(Shared, words) + 4 * kHold);
    if (e != cudaSuccess) return e;
    ready[f.dev].store(true, std::memory_order_relaxed);
  }
  const uint32_t S = sample_split(p.rows, p.vocab, f);
  p.split = log2_of(S);
  p.held = S * kHold >= p.vocab;
  p.ahead = std::max(1u, (uint32_t)f.sms / S);
  // (a block's batches are those of its warps in turn; or the weights of the row's batches)
  const uint32_t batches = (p.vocab + kBatch - 1) / kBatch, warps = S * kDrawWarps;
  const uint32_t words = p.held ? (batches + warps - 1) / warps * kDrawWarps * kBatch : 2 * batches;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.rows * S);
  cfg.blockDim = dim3(kDrawThreads);
  cfg.dynamicSmemBytes = offsetof(Shared, words) + 4 * words;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = S;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_sample_rows, p);
}

}  // namespace
}  // namespace ck

using namespace ck;

extern "C" {

uint32_t ck_host_sample_place(uint32_t distance, uint32_t temperature) {
  const uint32_t t = std::min(std::max(temperature, 1u), kMaxTemperature);
  return place_of(distance, places_of(t));
}

int ck_sample(const int64_t* dev_logits, size_t logits_stride, uint32_t rows, uint32_t vocab,
              const uint32_t* dev_temperature, const uint32_t* dev_top_k, const uint32_t* dev_top_p,
              const uint32_t* dev_min_p, const uint64_t* dev_random, const uint32_t* dev_exp, uint32_t* dev_token,
              uint32_t* dev_prob, uint32_t* dev_kept, void* stream) {
  if (rows < 1 || rows > 65536 || vocab < 1 || vocab > (1u << 20) || logits_stride < vocab || logits_stride >> 40)
    return CK_INVALID_ARGUMENT;
  if (!dev_logits || !dev_temperature || !dev_random || !dev_exp || !dev_token || !dev_prob || !dev_kept)
    return CK_INVALID_ARGUMENT;
  const void* in[] = {dev_logits, dev_random, dev_temperature, dev_top_k, dev_top_p, dev_min_p, dev_exp};
  const uint64_t r4 = 4ull * rows;
  const uint64_t in_bytes[] = {8 * ((rows - 1ull) * logits_stride + vocab), 8ull * rows, r4, dev_top_k ? r4 : 0,
                               dev_top_p ? r4 : 0, dev_min_p ? r4 : 0, 4 * 4097};
  const void* out[] = {dev_token, dev_prob, dev_kept};
  for (int i = 0; i < 7; ++i)
    if (!aligned_to(in[i], i < 2 ? 8 : 4)) return CK_INVALID_ARGUMENT;
  for (int o = 0; o < 3; ++o) {
    if (!aligned_to(out[o], 4)) return CK_INVALID_ARGUMENT;
    for (int i = 0; i < 7; ++i)
      if (overlaps(out[o], r4, in[i], in_bytes[i])) return CK_INVALID_ARGUMENT;
    for (int i = 0; i < o; ++i)
      if (overlaps(out[o], r4, out[i], r4)) return CK_INVALID_ARGUMENT;
  }
  const SampleParams p = {dev_logits, logits_stride, rows, vocab, dev_temperature, dev_top_k, dev_top_p, dev_min_p,
                          dev_random, dev_exp, dev_token, dev_prob, dev_kept, 0, 0, 0};
  CKP_CUDA(launch_sample(p, static_cast<cudaStream_t>(stream)));
  return CK_OK;
}

}  // extern "C"
