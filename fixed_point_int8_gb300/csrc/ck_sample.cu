// Sampling of many rows ("Sampling", the sum and draw passes) with a temperature, top-k, nucleus
// and least-probability filters, and given random numbers.
//
// With D the distance to the row's largest logit and i = floor(256 D / temperature) its place in the
// exponential table (4096 from 16 on), every filter keeps a beginning of the order by (D, token), and all
// tokens of a place weigh the same.  So the counts of the 4,097 places give everything but the
// boundary: the sums of top-k's tokens, how many tokens reach the nucleus, and the place at whose
// tokens the kept ones end, of which the nearest are then chosen by (D, token).  The draw walks
// the kept tokens in the order of the vocabulary, by each warp's sums.
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
  uint32_t split;  // blocks of a row's cluster
};

constexpr int kDrawThreads = 512, kDrawWarps = kDrawThreads / 32;
constexpr int kDrawBlocks = 2;                             // resident on an SM
constexpr uint32_t kPer = 16, kBatch = 32 * kPer;          // tokens a lane takes at once, and a warp
constexpr uint32_t kMaxBatches = (1u << 20) / kBatch;
constexpr uint32_t kBins = 4097, kMine = 9;                // places, and those a thread adds up
constexpr uint32_t kRoom = kMine * kDrawThreads;
constexpr uint32_t kList = 256;                            // tokens at the boundary that are ranked by counting
constexpr uint32_t kMaxSplit = 8;
constexpr uint32_t kOneQ24 = 1u << 24;
constexpr unsigned long long kNoBound = ~0ull;
static_assert(kRoom >= kBins && kMaxBatches * 8 <= kRoom * 4 && kList <= kDrawThreads, "shared memory");

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
__device__ __forceinline__ uint32_t remote_u32(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ void put_u64(const void* p, uint32_t rank, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(remote(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void put_u32(const void* p, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote(p, rank)), "r"(v) : "memory");
}
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

// A cluster of blocks a row (one block, where rows fill the GPU), warps taking batches of 512 tokens
// in turn.  The logits are read in each pass: the first from HBM, the next from L2.  Rows whose logits fit
// 32 bits (any that are not masked, in practice) go through them as 32-bit words.
struct Shared {
  uint32_t hist[kRoom];   // counts of this block; later the weights that are kept, by batch
  uint32_t full[kRoom];   // counts of the row
  uint32_t table[kRoom];  // the exponentials
  unsigned long long near_d[kList];
  uint32_t near_i[kList], n_near;
  unsigned long long red[kDrawWarps], peak, found[3];
  uint32_t red_c[kDrawWarps], red_i[kDrawWarps], least, tokens, wide;
  uint32_t f_place, f_count, f_rest;
  Places places;
};

// What is kept: tokens nearer than `first`, and of those from there to `last` the ones up to (d, token).
struct Bound {
  unsigned long long first, last, d;
  uint32_t token;
};

template <bool WIDE>
__device__ __forceinline__ void sample_row(const SampleParams& p, Shared& sm, long long m, uint32_t t, uint32_t top_k,
                                           uint32_t top_p, uint32_t min_p, bool filtered) {
  const uint32_t S = p.split, rank = blockIdx.x % S, row = blockIdx.x / S;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long* l = reinterpret_cast<const long long*>(p.logits) + (size_t)row * p.stride;
  const uint32_t batches = (p.vocab + kBatch - 1) / kBatch;
  using Word = typename std::conditional<WIDE, long long, int32_t>::type;
  using Distance = typename std::conditional<WIDE, unsigned long long, uint32_t>::type;
  auto word = [&](uint32_t i) -> Word {  // (of a narrow logit its low half)
    return WIDE ? (Word)__ldg(l + i) : (Word)__ldg(reinterpret_cast<const int32_t*>(l + i));
  };
  auto distance = [&](Word x) -> Distance { return (Distance)m - (Distance)x; };
  auto there = [&](Word x) { return !WIDE || x != (Word)LLONG_MIN; };
  const Places places = sm.places;
  auto place = [&](Distance d) { return place_of(WIDE && d >> 31 ? 0x7FFFFFFFu : (uint32_t)d, places); };
  // every batch of this warp: f(its number, its first token, whether it is whole, its words)
  auto each_batch = [&](auto f) {
    for (uint32_t b = rank * kDrawWarps + warp; b < batches; b += S * kDrawWarps) {
      const uint32_t i0 = b * kBatch + lane;
      Word x[kPer];
      if (b * kBatch + kBatch <= p.vocab) {
#pragma unroll
        for (uint32_t j = 0; j < kPer; ++j) x[j] = word(i0 + 32 * j);
        f(b, i0, true, x);
      } else {
#pragma unroll
        for (uint32_t j = 0; j < kPer; ++j) x[j] = i0 + 32 * j < p.vocab ? word(i0 + 32 * j) : 0;
        f(b, i0, false, x);
      }
    }
  };
  // every token of this thread that is not masked: f(distance, token)
  auto each = [&](auto f) {
    each_batch([&](uint32_t, uint32_t i0, bool whole, Word (&x)[kPer]) {
#pragma unroll
      for (uint32_t j = 0; j < kPer; ++j)
        if ((whole || i0 + 32 * j < p.vocab) && there(x[j])) f(distance(x[j]), i0 + 32 * j);
    });
  };

  if (t == 0) {  // the first largest
    uint32_t at = 0xFFFFFFFFu;
    each([&](Distance d, uint32_t i) {
      if (d == 0) at = min(at, i);
    });
    at = __reduce_min_sync(0xffffffffu, at);
    if (lane == 0) {
      if (S > 1)
        asm volatile("red.shared::cluster.min.u32 [%0], %1;" ::"r"(remote(&sm.least, 0)), "r"(at) : "memory");
      else
        atomicMin(&sm.least, at);
    }
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
  const uint32_t* full = S > 1 ? sm.full : sm.hist;
  if (filtered) {
    // the row's counts of the buckets that f names
    auto count_all = [&](auto f) {
      uint32_t last = 0;
      each([&](Distance d, uint32_t i) {
        const uint32_t b = f(d, i);
        if (b < kBins - 1)
          atomicAdd(sm.hist + b, 1u);
        else
          last += b == kBins - 1;  // (often most of them)
      });
      last = __reduce_add_sync(0xffffffffu, last);
      if (lane == 0 && last) atomicAdd(sm.hist + kBins - 1, last);
      row_sync(S);
      if (S == 1) return;
      const uint32_t width = (kRoom + S - 1) / S, b1 = min(kRoom, (rank + 1) * width);
      for (uint32_t b = rank * width + tid; b < b1; b += kDrawThreads) {
        uint32_t part[kMaxSplit], c = 0;
#pragma unroll
        for (uint32_t k = 0; k < kMaxSplit; ++k) part[k] = k < S ? remote_u32(sm.hist + b, k) : 0;
#pragma unroll
        for (uint32_t k = 0; k < kMaxSplit; ++k) c += part[k];
        for (uint32_t k = 0; k < S; ++k) put_u32(sm.full + b, k, c);
      }
      row_sync(S);
    };
    count_all([&](Distance d, uint32_t) { return place(d); });
    // counts and weights before this thread's places
    const uint32_t b0 = tid * kMine;
    uint32_t mine = 0, near = 0;
    unsigned long long heavy = 0;
    const unsigned long long least_w = (unsigned long long)min_p * sm.table[0];
#pragma unroll
    for (uint32_t j = 0; j < kMine; ++j) {
      const uint32_t c = full[b0 + j], e = sm.table[b0 + j];
      mine += c;
      heavy += (unsigned long long)c * e;
      if ((unsigned long long)e << 24 >= least_w) near += c;
    }
    const uint32_t count_in = (uint32_t)warp_inclusive_scan((unsigned long long)mine, lane);
    const unsigned long long weight_in = warp_inclusive_scan(heavy, lane);
    near = __reduce_add_sync(0xffffffffu, near);
    if (lane == 31) {
      sm.red_c[warp] = count_in;
      sm.red[warp] = weight_in;
      sm.red_i[warp] = near;
    }
    __syncthreads();
    uint32_t before = count_in - mine, total = 0;
    unsigned long long weight = weight_in - heavy, z = 0;
    near = 0;
#pragma unroll
    for (uint32_t w = 0; w < kDrawWarps; ++w) {
      if (w < warp) {
        before += sm.red_c[w];
        weight += sm.red[w];
      }
      total += sm.red_c[w];
      z += sm.red[w];
      near += sm.red_i[w];
    }
    uint32_t keep = top_k ? min(top_k, total) : total;
    if (top_p < kOneQ24) {
      if (keep < total) {  // the weight of the first `keep`
        if (before < keep && keep <= before + mine) {
          uint32_t c = before;
          unsigned long long w = weight;
          for (uint32_t j = 0; j < kMine; ++j) {
            const uint32_t take = min(full[b0 + j], keep - c);
            w += (unsigned long long)take * sm.table[b0 + j];
            c += take;
          }
          sm.found[0] = w;
        }
        __syncthreads();
        z = sm.found[0];
      }
      const unsigned long long target = (z >> 24) * top_p + (((z & (kOneQ24 - 1)) * top_p) >> 24);
      if (tid == 0 && target == 0) sm.found[1] = 1;
      if (weight < target && target <= weight + heavy) {
        uint32_t c = before;
        unsigned long long w = weight;
        for (uint32_t j = 0; j < kMine; ++j) {
          const unsigned long long here = (unsigned long long)full[b0 + j] * sm.table[b0 + j];
          if (w + here >= target) {
            sm.found[1] = c + (target - w + sm.table[b0 + j] - 1) / sm.table[b0 + j];
            break;
          }
          w += here;
          c += full[b0 + j];
        }
      }
      __syncthreads();
      keep = min(keep, (uint32_t)sm.found[1]);
    }
    if (min_p) keep = max(1u, min(keep, near));
    // the place at which the kept ones end, and how many of it
    if (before < keep && keep <= before + mine) {
      uint32_t c = before, j = 0;
      while (c + full[b0 + j] < keep) c += full[b0 + j++];
      sm.f_place = b0 + j;
      sm.f_count = full[b0 + j];
      sm.f_rest = keep - c;
    }
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
        if (by_token && t_span == 1) break;  // (one token at one distance: not reached)
        const unsigned long long range = by_token ? t_span : span;
        uint32_t shift = 0;
        while (((range - 1) >> shift) >= 4096) ++shift;
        __syncthreads();  // the counts have been read
        for (uint32_t i = tid; i < kRoom; i += kDrawThreads) sm.hist[i] = 0;
        __syncthreads();
        count_all([&](Distance d, uint32_t i) {
          const unsigned long long at = by_token ? i - t_lo : d - lo;
          if (d < lo || d - lo >= span || (by_token && (i < t_lo || at >= t_span))) return kBins;
          return tail ? tail_bucket(at) : (uint32_t)(at >> shift);
        });
        uint32_t own = 0;
        for (uint32_t j = 0; j < kMine; ++j) own += full[b0 + j];
        const uint32_t upto = (uint32_t)warp_inclusive_scan((unsigned long long)own, lane);
        if (lane == 31) sm.red_c[warp] = upto;
        __syncthreads();
        uint32_t c = upto - own;
        for (uint32_t w = 0; w < warp; ++w) c += sm.red_c[w];
        if (c < rest && rest <= c + own) {
          uint32_t j = 0;
          while (c + full[b0 + j] < rest) c += full[b0 + j++];
          sm.f_place = b0 + j;
          sm.f_count = full[b0 + j];
          sm.f_rest = rest - c;
        }
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
    if (S == 1) __syncthreads();  // (the counts have been read: the weights by batch take their place)
  }

  // ---- the weights that are kept, by batch, and the tokens at the boundary: all to the first block
  unsigned long long* weights = reinterpret_cast<unsigned long long*>(sm.hist);
  uint32_t tokens = 0;
  each_batch([&](uint32_t b, uint32_t i0, bool whole, Word (&x)[kPer]) {
    unsigned long long sum = 0;
#pragma unroll
    for (uint32_t j = 0; j < kPer; ++j) {
      if ((!whole && i0 + 32 * j >= p.vocab) || !there(x[j])) continue;
      const Distance d = distance(x[j]);
      if (!filtered) {
        sum += sm.table[place(d)];
        if (WIDE) ++tokens;
      } else if (d <= bound.last) {
        if (d < bound.first || (!listed && (d < bound.d || (d == bound.d && i0 + 32 * j <= bound.token)))) {
          sum += sm.table[place(d)];
        } else if (listed) {
          const uint32_t to = S > 1 ? remote_count(&sm.n_near, 0) : atomicAdd(&sm.n_near, 1u);
          if (S > 1) {
            put_u64(sm.near_d + to, 0, d);
            put_u32(sm.near_i + to, 0, i0 + 32 * j);
          } else {
            sm.near_d[to] = d;
            sm.near_i[to] = i0 + 32 * j;
          }
        }
      }
    }
    if (!filtered || __any_sync(0xffffffffu, sum != 0)) sum = warp_sum34(sum);
    if (lane == 0) {
      if (S > 1)
        put_u64(weights + b, 0, sum);
      else
        weights[b] = sum;
    }
  });
  if (WIDE && !filtered) {
    tokens = __reduce_add_sync(0xffffffffu, tokens);
    if (lane == 0) {
      if (S > 1)
        asm volatile("red.shared::cluster.add.u32 [%0], %1;" ::"r"(remote(&sm.tokens, 0)), "r"(tokens) : "memory");
      else
        atomicAdd(&sm.tokens, tokens);
    }
  }
  row_sync(S);
  if (rank != 0) return;
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
  if (warp != 0) return;
  // ---- the draw, by the first warp: the lane whose batches hold it, the batch, its 32 tokens, the token
  const uint32_t own = (batches + 31) / 32, g0 = min(batches, lane * own), g1 = min(batches, g0 + own);
  unsigned long long sum = 0;
  for (uint32_t g = g0; g < g1; ++g) sum += weights[g];
  const unsigned long long upto = warp_inclusive_scan(sum, lane), z = __shfl_sync(0xffffffffu, upto, 31);
  if (z == 0) {  // (a table of zeros)
    if (lane == 0) {
      p.token[row] = CK_NO_TOKEN;
      p.prob[row] = 0;
      p.kept[row] = 0;
    }
    return;
  }
  const unsigned long long draw = p.random[row] % z;
  const int holder = __ffs((int)__ballot_sync(0xffffffffu, upto > draw)) - 1;
  unsigned long long rem = draw - __shfl_sync(0xffffffffu, upto - sum, holder);
  uint32_t batch = g0;
  if ((int)lane == holder)
    while (rem >= weights[batch]) rem -= weights[batch++];
  rem = __shfl_sync(0xffffffffu, rem, holder);
  batch = __shfl_sync(0xffffffffu, batch, holder);
  const uint32_t i0 = batch * kBatch + lane;
  uint32_t e[kPer];
#pragma unroll
  for (uint32_t j = 0; j < kPer; ++j) {
    const uint32_t i = i0 + 32 * j;
    const Word x = i < p.vocab ? word(i) : 0;
    const Distance d = distance(x);
    const bool in = i < p.vocab && there(x) &&
                    (!filtered || d < bound.first || (d <= bound.last && (d < bound.d || (d == bound.d && i <= bound.token))));
    e[j] = in ? sm.table[place(d)] : 0;
  }
#pragma unroll
  for (uint32_t j = 0; j < kPer; ++j) {
    const unsigned long long here = warp_sum34(e[j]);
    if (rem < here) {
      const unsigned long long to = warp_inclusive_scan((unsigned long long)e[j], lane);
      if (lane == (uint32_t)__ffs((int)__ballot_sync(0xffffffffu, to > rem)) - 1) {
        p.token[row] = i0 + 32 * j;
        p.prob[row] = (uint32_t)(((unsigned long long)e[j] << 24) / z);
        p.kept[row] = filtered ? kept : WIDE ? sm.tokens : p.vocab;
      }
      return;
    }
    rem -= here;
  }
}

__global__ void __launch_bounds__(kDrawThreads, kDrawBlocks) k_sample_rows(const SampleParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sm = *reinterpret_cast<Shared*>(smem);
  const uint32_t S = p.split, rank = blockIdx.x % S, row = blockIdx.x / S;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long* l = reinterpret_cast<const long long*>(p.logits) + (size_t)row * p.stride;
  const uint32_t batches = (p.vocab + kBatch - 1) / kBatch;
  const uint32_t t = p.temperature[row];
  const uint32_t top_k = p.top_k ? p.top_k[row] : 0, top_p = p.top_p ? min(p.top_p[row], kOneQ24) : kOneQ24;
  const uint32_t min_p = p.min_p ? min(p.min_p[row], kOneQ24) : 0;
  const bool filtered = (top_k != 0 && top_k < p.vocab) || top_p < kOneQ24 || min_p != 0;
  // ---- the largest logit, of 32 bits, and whether any has more
  int32_t m32 = INT32_MIN, more = 0;
  for (uint32_t b = rank * kDrawWarps + warp; b < batches; b += S * kDrawWarps) {
    const uint32_t i0 = b * kBatch + lane;
    long long x[kPer];
#pragma unroll
    for (uint32_t j = 0; j < kPer; ++j) x[j] = i0 + 32 * j < p.vocab ? __ldg(l + i0 + 32 * j) : (long long)INT32_MIN;
#pragma unroll
    for (uint32_t j = 0; j < kPer; ++j) {
      m32 = max(m32, (int32_t)x[j]);
      more |= (int32_t)(x[j] >> 32) ^ ((int32_t)x[j] >> 31);
    }
  }
  for (uint32_t i = tid; i < kRoom; i += kDrawThreads) {
    sm.hist[i] = 0;
    sm.table[i] = i < kBins ? min(__ldg(p.exp_tab + i), 1u << 30) : 0;
  }
  if (tid == 0) {
    sm.n_near = 0;
    sm.tokens = 0;
    sm.least = 0xFFFFFFFFu;
    if (t != 0 && t <= kMaxTemperature) sm.places = places_of(t);
  }
  m32 = __reduce_max_sync(0xffffffffu, m32);
  if (lane == 0) sm.red_i[warp] = (uint32_t)m32;
  bool wide = __syncthreads_or(more);
#pragma unroll
  for (int w = 0; w < kDrawWarps; ++w) m32 = max(m32, (int32_t)sm.red_i[w]);
  if (tid == 0) sm.peak = (unsigned long long)(uint32_t)m32 | (unsigned long long)wide << 32;
  row_sync(S);
  for (uint32_t k = 0; S > 1 && k < S; ++k) {
    const unsigned long long other = remote_u64(&sm.peak, k);
    m32 = max(m32, (int32_t)other);
    wide |= other >> 32 != 0;
  }
  if (t > kMaxTemperature) {
    row_sync(S);
    if (rank == 0 && tid == 0) {
      p.token[row] = CK_NO_TOKEN;
      p.prob[row] = 0;
      p.kept[row] = 0;
    }
    return;
  }
  if (!wide) {
    sample_row<false>(p, sm, m32, t, top_k, top_p, min_p, filtered);
    return;
  }
  // ---- the largest of 64 bits
  row_sync(S);  // the 32-bit ones have been read
  long long m = LLONG_MIN;
  for (uint32_t b = rank * kDrawWarps + warp; b < batches; b += S * kDrawWarps)
#pragma unroll
    for (uint32_t j = 0; j < kPer; ++j) {
      const uint32_t i = b * kBatch + lane + 32 * j;
      m = max(m, i < p.vocab ? __ldg(l + i) : LLONG_MIN);
    }
  m = warp_max(m);
  if (lane == 0) sm.red[warp] = (unsigned long long)m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kDrawWarps; ++w) m = max(m, (long long)sm.red[w]);
  if (tid == 0) sm.peak = (unsigned long long)m;
  row_sync(S);
  for (uint32_t k = 0; S > 1 && k < S; ++k) m = max(m, (long long)remote_u64(&sm.peak, k));
  if (m == LLONG_MIN) {  // every token is masked
    row_sync(S);
    if (rank == 0 && tid == 0) {
      p.token[row] = CK_NO_TOKEN;
      p.prob[row] = 0;
      p.kept[row] = 0;
    }
    return;
  }
  sample_row<true>(p, sm, m, t, top_k, top_p, min_p, filtered);
}

// Blocks of a row's cluster: as many as there are SMs for every row, of at least a batch a warp.
uint32_t sample_split(uint32_t rows, uint32_t vocab, const DeviceFacts& f) {
  uint32_t S = 1;
  while (S < kMaxSplit && 2ull * S * rows <= (uint64_t)f.sms && 2 * S * kDrawWarps * kBatch <= 2 * vocab) S *= 2;
  return S;
}

cudaError_t launch_sample(SampleParams p, cudaStream_t s) {
  DeviceFacts f;
  cudaError_t e = device_facts(&f);
  if (e != cudaSuccess) return e;
  static std::atomic<bool> ready[64];
  if (!ready[f.dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(k_sample_rows, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Shared));
    if (e != cudaSuccess) return e;
    ready[f.dev].store(true, std::memory_order_relaxed);
  }
  p.split = sample_split(p.rows, p.vocab, f);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.rows * p.split);
  cfg.blockDim = dim3(kDrawThreads);
  cfg.dynamicSmemBytes = sizeof(Shared);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.split;
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
                          dev_random, dev_exp, dev_token, dev_prob, dev_kept, 1};
  CKP_CUDA(launch_sample(p, static_cast<cudaStream_t>(stream)));
  return CK_OK;
}

}  // extern "C"
