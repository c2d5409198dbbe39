// Sampling of many rows ("Sampling", the sum and draw passes) with a temperature, top-k, nucleus
// and least-probability filters, and given random numbers.
//
// With D the distance to the row's largest logit and i = floor(256 D / temperature) its place in the
// exponential table (4096 from 16 on), every filter keeps a beginning of the order by (D, token), and all
// tokens of a place weigh the same.  So the counts of the 4,097 places give everything but the
// boundary: the sums of top-k's tokens, how many tokens reach the nucleus, and the place at whose
// tokens the kept ones end, of which the nearest are then chosen by (D, token).  The draw walks
// the kept tokens in the order of the vocabulary, by each warp's sums.
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

constexpr int kDrawThreads = 256, kDrawWarps = kDrawThreads / 32;
constexpr uint32_t kPer = 16;                              // logits a thread holds
constexpr uint32_t kHold = kPer * kDrawThreads;            // and a block
constexpr uint32_t kBins = 4097, kMine = 17;               // places, and those a thread adds up
constexpr uint32_t kRoom = kMine * kDrawThreads;
constexpr uint32_t kList = 256;                            // tokens at the boundary that are ranked by counting
constexpr uint32_t kMaxSplit = 8;
constexpr uint32_t kOneQ24 = 1u << 24;
// distances held in 32 bits: a masked token (or none), and one to be read again
constexpr uint32_t kMasked = 0xFFFFFFFFu, kFar = 0xFFFFFFFEu;
constexpr unsigned long long kNoBound = ~0ull;

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
__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The place of a distance below 16 temperatures: floor(256 d / t) by the reciprocal r = floor(2^32
// / t) (2^32 - 1 for t = 1), short of the quotient by less than one.
__host__ __device__ __forceinline__ uint32_t reciprocal_of(uint32_t t) {
  return t > 1 ? (uint32_t)((1ull << 32) / t) : 0xFFFFFFFFu;
}
__host__ __device__ __forceinline__ uint32_t place_of(uint32_t d, uint32_t t, uint32_t r) {
  if (d >= 16 * t) return 4096;
  const uint32_t n = d << 8;
#ifdef __CUDA_ARCH__
  const uint32_t q = __umulhi(n, r);
#else
  const uint32_t q = (uint32_t)(((uint64_t)n * r) >> 32);
#endif
  return q + (n - q * t >= t);
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

// What is kept: tokens nearer than d, and those at d up to the token.
struct Bound {
  unsigned long long d;
  uint32_t token;
};

template <bool ONE>
__global__ void __launch_bounds__(kDrawThreads) k_sample_rows(const SampleParams p) {
  __shared__ uint32_t hist[kRoom], full[kRoom];
  __shared__ unsigned long long near_d[kList];
  __shared__ uint32_t near_i[kList], n_near;
  __shared__ unsigned long long sums[kMaxSplit * kDrawWarps], red[kDrawWarps], peak, found[3];
  __shared__ uint32_t counts[kMaxSplit * kDrawWarps], red_c[kDrawWarps], red_i[kDrawWarps], least;
  __shared__ uint32_t f_place, f_count, f_rest;
  const uint32_t S = p.split, rank = blockIdx.x % S, row = blockIdx.x / S;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t per = (p.vocab + S - 1) / S, v0 = min(p.vocab, rank * per), n = min(p.vocab, v0 + per) - v0;
  // a warp's tokens follow one another
  const uint32_t each = ((n + kDrawWarps - 1) / kDrawWarps + 31) & ~31u, w0 = min(n, warp * each), wn = min(n, w0 + each) - w0;
  const long long* l = reinterpret_cast<const long long*>(p.logits) + (size_t)row * p.stride + v0 + w0;
  const uint32_t first = v0 + w0;  // the warp's first token

  long long x[kPer];
  auto load = [&](uint32_t base) {
#pragma unroll
    for (uint32_t j = 0; j < kPer; ++j) {
      const uint32_t i = base + 32 * j + lane;
      x[j] = i < wn ? __ldg(l + i) : LLONG_MIN;
    }
  };
  if (ONE) load(0);
  const uint32_t t = p.temperature[row];
  const uint32_t top_k = p.top_k ? p.top_k[row] : 0, top_p = p.top_p ? min(p.top_p[row], kOneQ24) : kOneQ24;
  const uint32_t min_p = p.min_p ? min(p.min_p[row], kOneQ24) : 0;
  const bool filtered = (top_k != 0 && top_k < p.vocab) || top_p < kOneQ24 || min_p != 0;
  auto weight_at = [&](uint32_t place) { return min(__ldg(p.exp_tab + place), 1u << 30); };
  for (uint32_t i = tid; i < kRoom; i += kDrawThreads) hist[i] = filtered || i >= kBins ? 0 : weight_at(i);
  if (tid == 0) n_near = 0;

  // ---- the largest logit
  long long m = LLONG_MIN;
  for (uint32_t base = 0; base < (ONE ? 1 : wn); base += 32 * kPer) {
    if (!ONE) load(base);
#pragma unroll
    for (uint32_t j = 0; j < kPer; ++j) m = max(m, x[j]);
  }
  m = warp_max(m);
  if (lane == 0) red[warp] = (unsigned long long)m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kDrawWarps; ++w) m = max(m, (long long)red[w]);
  if (tid == 0) peak = (unsigned long long)m;
  row_sync(S);
  for (uint32_t k = 0; S > 1 && k < S; ++k) m = max(m, (long long)remote_u64(&peak, k));
  if (m == LLONG_MIN || t > kMaxTemperature) {  // nothing to choose from (for every block of the row)
    row_sync(S);
    if (rank == 0 && tid == 0) {
      p.token[row] = CK_NO_TOKEN;
      p.prob[row] = 0;
      p.kept[row] = 0;
    }
    return;
  }

  // ---- distances, in 32 bits
  uint32_t d[kPer];
  auto distances = [&] {
#pragma unroll
    for (uint32_t j = 0; j < kPer; ++j) {
      const unsigned long long w = (unsigned long long)m - (unsigned long long)x[j];
      d[j] = x[j] == LLONG_MIN ? kMasked : w < kFar ? (uint32_t)w : kFar;
    }
  };
  if (ONE) distances();
  // every token of this thread that is not masked: f(distance in 32 bits, its number in the warp)
  auto all = [&](auto f) {
    for (uint32_t base = 0; base < (ONE ? 1 : wn); base += 32 * kPer) {
      if (!ONE) {
        load(base);
        distances();
      }
#pragma unroll
      for (uint32_t j = 0; j < kPer; ++j)
        if (d[j] != kMasked) f(d[j], base + 32 * j + lane);
    }
  };
  auto exact = [&](uint32_t w, uint32_t i) {
    return w != kFar ? (unsigned long long)w : (unsigned long long)m - (unsigned long long)__ldg(l + i);
  };

  if (t == 0) {  // the first largest
    uint32_t at = 0xFFFFFFFFu;
    all([&](uint32_t w, uint32_t i) {
      if (w == 0) at = min(at, first + i);
    });
    at = __reduce_min_sync(0xffffffffu, at);
    if (lane == 0) red_i[warp] = at;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kDrawWarps; ++w) at = min(at, red_i[w]);
    if (tid == 0) least = at;
    row_sync(S);
    if (rank == 0) {
      for (uint32_t k = 0; S > 1 && k < S; ++k) at = min(at, remote_u32(&least, k));
      if (tid == 0) {
        p.token[row] = at;
        p.prob[row] = kOneQ24;
        p.kept[row] = 1;
      }
    }
    row_sync(S);  // no block leaves while another reads its minimum
    return;
  }
  const uint32_t rt = reciprocal_of(t);

  Bound bound = {kNoBound, 0xFFFFFFFFu};
  uint32_t kept = 0;
  if (filtered) {
    // the row's counts of the buckets that f names, in every block's `full`
    auto count_all = [&](auto f) {
      uint32_t last = 0;
      all([&](uint32_t w, uint32_t i) {
        const uint32_t b = f(w, i);
        if (b == kBins - 1)
          ++last;  // (often most of them)
        else if (b < kBins)
          atomicAdd(hist + b, 1u);
      });
      last = __reduce_add_sync(0xffffffffu, last);
      if (lane == 0 && last) atomicAdd(hist + kBins - 1, last);
      row_sync(S);
      const uint32_t width = (kBins + S - 1) / S, b1 = min(kBins, (rank + 1) * width);
      for (uint32_t b = rank * width + tid; b < b1; b += kDrawThreads) {
        uint32_t part[kMaxSplit], c = 0;
#pragma unroll
        for (uint32_t k = 0; k < kMaxSplit; ++k) part[k] = k < S ? (S > 1 ? remote_u32(hist + b, k) : hist[b]) : 0;
#pragma unroll
        for (uint32_t k = 0; k < kMaxSplit; ++k) c += part[k];
        for (uint32_t k = 0; k < S; ++k)
          if (S > 1)
            put_u32(full + b, k, c);
          else
            full[b] = c;
      }
      for (uint32_t b = kBins + tid; b < kRoom; b += kDrawThreads) full[b] = 0;
      row_sync(S);
    };
    count_all([&](uint32_t w, uint32_t) { return place_of(w, t, rt); });
    for (uint32_t i = tid; i < kBins; i += kDrawThreads) hist[i] = weight_at(i);
    __syncthreads();
    // counts and weights before this thread's places
    const uint32_t b0 = tid * kMine;
    uint32_t mine = 0, near = 0;
    unsigned long long heavy = 0;
    const unsigned long long least_w = (unsigned long long)min_p * hist[0];
#pragma unroll
    for (uint32_t j = 0; j < kMine; ++j) {
      const uint32_t c = full[b0 + j], e = b0 + j < kBins ? hist[b0 + j] : 0;
      mine += c;
      heavy += (unsigned long long)c * e;
      if ((unsigned long long)e << 24 >= least_w) near += c;
    }
    const uint32_t count_in = (uint32_t)warp_inclusive_scan((unsigned long long)mine, lane);
    const unsigned long long weight_in = warp_inclusive_scan(heavy, lane);
    near = __reduce_add_sync(0xffffffffu, near);
    if (lane == 31) {
      red_c[warp] = count_in;
      red[warp] = weight_in;
      red_i[warp] = near;
    }
    __syncthreads();
    uint32_t before = count_in - mine, total = 0;
    unsigned long long weight = weight_in - heavy, z = 0;
    near = 0;
#pragma unroll
    for (uint32_t w = 0; w < kDrawWarps; ++w) {
      if (w < warp) {
        before += red_c[w];
        weight += red[w];
      }
      total += red_c[w];
      z += red[w];
      near += red_i[w];
    }
    uint32_t keep = top_k ? min(top_k, total) : total;
    if (top_p < kOneQ24) {
      if (keep < total) {  // the weight of the first `keep`
        if (before < keep && keep <= before + mine) {
          uint32_t c = before;
          unsigned long long w = weight;
          for (uint32_t j = 0; j < kMine; ++j) {
            const uint32_t take = min(full[b0 + j], keep - c);
            w += (unsigned long long)take * hist[b0 + j];
            c += take;
          }
          found[0] = w;
        }
        __syncthreads();
        z = found[0];
      }
      const unsigned long long target = (z >> 24) * top_p + (((z & (kOneQ24 - 1)) * top_p) >> 24);
      if (tid == 0) found[1] = 1;  // (a target of zero)
      __syncthreads();
      if (weight < target && target <= weight + heavy) {
        uint32_t c = before;
        unsigned long long w = weight;
        for (uint32_t j = 0; j < kMine; ++j) {
          const unsigned long long here = (unsigned long long)full[b0 + j] * hist[b0 + j];
          if (w + here >= target) {
            found[1] = c + (target - w + hist[b0 + j] - 1) / hist[b0 + j];
            break;
          }
          w += here;
          c += full[b0 + j];
        }
      }
      __syncthreads();
      keep = min(keep, (uint32_t)found[1]);
    }
    if (min_p) keep = max(1u, min(keep, near));
    // the place at which the kept ones end, and how many of it
    if (before < keep && keep <= before + mine) {
      uint32_t c = before, j = 0;
      while (c + full[b0 + j] < keep) c += full[b0 + j++];
      f_place = b0 + j;
      f_count = full[b0 + j];
      f_rest = keep - c;
    }
    __syncthreads();
    kept = keep;
    const uint32_t place = f_place;
    uint32_t among = f_count, rest = f_rest;
    unsigned long long lo = first_of(place, t), span = place < 4096 ? first_of(place + 1, t) - lo : 0 - lo;  // (2^64 - lo)
    bound.d = place < 4096 ? lo + span - 1 : kNoBound;
    // the nearest `rest` of the `among` at distances lo .. lo + span - 1, by distance and then by token
    bool by_token = false, tail = place == 4096;
    uint32_t t_lo = 0, t_span = p.vocab;
    while (rest < among) {
      if (!by_token && span == 1) by_token = true;
      auto in = [&](uint32_t w, uint32_t i, unsigned long long* at) {
        const unsigned long long e = exact(w, i);
        *at = by_token ? first + i - t_lo : e - lo;
        return e >= lo && e - lo < span && (!by_token || *at < t_span);
      };
      if (among <= kList) {
        all([&](uint32_t w, uint32_t i) {
          unsigned long long at;
          if (!in(w, i, &at)) return;
          const unsigned long long e = exact(w, i);
          const uint32_t to = S > 1 ? remote_count(&n_near, 0) : atomicAdd(&n_near, 1u);
          for (uint32_t k = 0; k < S; ++k) {
            if (S > 1) {
              put_u64(near_d + to, k, e);
              put_u32(near_i + to, k, first + i);
            } else {
              near_d[to] = e;
              near_i[to] = first + i;
            }
          }
        });
        row_sync(S);
        if (tid < among) {
          const unsigned long long e = near_d[tid];
          const uint32_t i = near_i[tid];
          uint32_t r = 0;
          for (uint32_t k = 0; k < among; ++k) r += near_d[k] < e || (near_d[k] == e && near_i[k] < i);
          if (r == rest - 1) {
            found[2] = e;
            least = i;
          }
        }
        __syncthreads();
        bound = {found[2], least};
        break;
      }
      // one more step towards it, in up to 4,096 buckets
      const unsigned long long range = by_token ? t_span : span;
      uint32_t shift = 0;
      while (((range - 1) >> shift) >= 4096) ++shift;
      for (uint32_t i = tid; i < kRoom; i += kDrawThreads) hist[i] = 0;
      __syncthreads();
      count_all([&](uint32_t w, uint32_t i) {
        unsigned long long at;
        if (!in(w, i, &at)) return kBins;
        return tail ? tail_bucket(at) : (uint32_t)(at >> shift);
      });
      uint32_t own = 0;
      for (uint32_t j = 0; j < kMine; ++j) own += full[b0 + j];
      const uint32_t upto = (uint32_t)warp_inclusive_scan((unsigned long long)own, lane);
      if (lane == 31) red_c[warp] = upto;
      __syncthreads();
      uint32_t c = upto - own;
      for (uint32_t w = 0; w < warp; ++w) c += red_c[w];
      if (c < rest && rest <= c + own) {
        uint32_t j = 0;
        while (c + full[b0 + j] < rest) c += full[b0 + j++];
        f_place = b0 + j;
        f_count = full[b0 + j];
        f_rest = rest - c;
      }
      __syncthreads();
      const uint32_t b = f_place;
      among = f_count;
      rest = f_rest;
      if (by_token) {
        t_lo += b << shift;
        t_span = min(1u << shift, t_span - (b << shift));
        bound.token = t_lo + t_span - 1;
        bound.d = lo;
      } else {
        const unsigned long long from = tail ? tail_first(b) : (unsigned long long)b << shift;
        const unsigned long long wide = tail ? (b < 64 ? 1ull : 1ull << ((b >> 6) - 1)) : 1ull << shift;
        span = min(wide, span - from);
        lo += from;
        bound.d = lo + span - 1;
        tail = false;
      }
      __syncthreads();
    }
  }

  // ---- the weights that are kept, by warp
  auto weight_of = [&](uint32_t w, uint32_t i) -> uint32_t {
    if (filtered) {
      const unsigned long long e = bound.d >= kFar ? exact(w, i) : w;
      if (e > bound.d || (e == bound.d && first + i > bound.token)) return 0;
      return weight_at(place_of(w, t, rt));
    }
    return hist[place_of(w, t, rt)];
  };
  unsigned long long sum = 0;
  uint32_t some = 0;
  all([&](uint32_t w, uint32_t i) {
    sum += weight_of(w, i);
    ++some;
  });
  sum = warp_sum(sum);
  some = __reduce_add_sync(0xffffffffu, some);
  if (lane < S) {  // to every block of the row
    if (S > 1) {
      put_u64(sums + rank * kDrawWarps + warp, lane, sum);
      put_u32(counts + rank * kDrawWarps + warp, lane, some);
    } else {
      sums[warp] = sum;
      counts[warp] = some;
    }
  }
  row_sync(S);
  unsigned long long z = 0, ahead = 0;
  uint32_t tokens = 0;
  for (uint32_t k = 0; k < S * kDrawWarps; ++k) {
    if (k < rank * kDrawWarps + warp) ahead += sums[k];
    z += sums[k];
    tokens += counts[k];
  }
  if (z == 0) {  // (a table of zeros)
    if (rank == 0 && tid == 0) {
      p.token[row] = CK_NO_TOKEN;
      p.prob[row] = 0;
      p.kept[row] = 0;
    }
    return;
  }
  const unsigned long long r = p.random[row] % z;
  if (r < ahead || r - ahead >= sum) return;
  // ---- this warp's tokens hold the draw
  unsigned long long rem = r - ahead;
  for (uint32_t i0 = 0; i0 < wn; i0 += 32) {
    const uint32_t i = i0 + lane;
    const long long y = i < wn ? __ldg(l + i) : LLONG_MIN;
    const unsigned long long w = (unsigned long long)m - (unsigned long long)y;
    const uint32_t e = y == LLONG_MIN ? 0 : weight_of(w < kFar ? (uint32_t)w : kFar, i);
    const unsigned long long upto = warp_inclusive_scan((unsigned long long)e, lane);
    const unsigned long long here = __shfl_sync(0xffffffffu, upto, 31);
    if (rem < here) {
      if (lane == (uint32_t)__ffs((int)__ballot_sync(0xffffffffu, upto > rem)) - 1) {
        p.token[row] = first + i;
        p.prob[row] = (uint32_t)(((unsigned long long)e << 24) / z);
        p.kept[row] = filtered ? kept : tokens;
      }
      return;
    }
    rem -= here;
  }
}

cudaError_t launch_sample(const SampleParams& p, cudaStream_t s) {
  k_sample_rows<false><<<p.rows, kDrawThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace ck

using namespace ck;

extern "C" {

uint32_t ck_host_sample_place(uint32_t distance, uint32_t temperature) {
  const uint32_t t = std::min(std::max(temperature, 1u), kMaxTemperature);
  return place_of(distance, t, reciprocal_of(t));
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
