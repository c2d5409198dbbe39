// Beam search's selection over beams and vocabulary ("Sampling", with the sum pass at
// temperature one): every beam's continuations by their distance to its largest logit, the
// logarithm of its sum of exponentials, and the best of all beams together.
#include "ck_paged.cuh"
#include "ck_tc.cuh"

namespace ck {
namespace {

constexpr long long kDeadScore = -(1ll << 61);
constexpr unsigned long long kMaxDistance = 1ull << 62;
constexpr unsigned long long kLost = ~0ull;  // a sum of exponentials (below 2^51) that is none
std::atomic<uint32_t> g_wait_limit{0};       // ck_set_beam_wait_limit

// ln(z / 2^30), 16 fraction bits (0 below 2^30): z = 2^n y with y in [1, 2), ln y = 2 atanh t
// of t = (y - 1) / (y + 1) <= 1/3, its series to t^15 (the next term is below 2^-28).
__host__ __device__ inline int64_t log_sum(uint64_t z) {
  if (z < (1ull << 30)) z = 1ull << 30;
#ifdef __CUDA_ARCH__
  const uint32_t n = 33 - (uint32_t)__clzll((long long)z);
#else
  const uint32_t n = 33 - (uint32_t)__builtin_clzll(z);
#endif
  const uint64_t y = z >> n, one = 1ull << 30;
  const uint64_t t = div_small_quotient((y - one) << 30, (uint32_t)(y + one)), T = (t * t) >> 30;
  uint64_t c = 71582788;
  c = 82595525 + ((c * T) >> 30);
  c = 97612893 + ((c * T) >> 30);
  c = 119304647 + ((c * T) >> 30);
  c = 153391689 + ((c * T) >> 30);
  c = 214748365 + ((c * T) >> 30);
  c = 357913941 + ((c * T) >> 30);
  c = 1073741824 + ((c * T) >> 30);
  return (int64_t)((n * 744261118ull + 2 * ((t * c) >> 30) + (1u << 13)) >> 14);
}

struct BeamParams {
  const int64_t* logits;
  size_t stride;
  uint32_t groups, beams, vocab, flags, done_token;
  const int64_t* scores;
  const uint8_t* done;
  const uint32_t* exp_tab;
  int64_t* scores_out;
  uint32_t* parent;
  uint32_t* token;
  uint8_t* done_out;
  // of every row and block of its cluster: the sum of exponentials, and the block's nearest
  // continuations, nearest first (distance all ones: none; token `vocab`: an ended beam)
  uint32_t split;
  uint32_t polls;                 // of a row's wait for the cluster's maxima, before it is given up
  unsigned long long* part_z;     // [rows][split]; kLost: the block gave the row up
  unsigned long long* list_d;     // [rows][split][beams]
  uint32_t* list_token;           // [rows][split][beams]
};

constexpr int kBeamThreads = 256, kBeamWarps = kBeamThreads / 32;
constexpr int kBeamBlocks = 5;                           // resident on an SM
constexpr int kPer = 16;                                 // logits a thread holds
constexpr uint32_t kRound = kPer * kBeamThreads;         // logits a block takes at once
constexpr uint32_t kFound = 512;                         // continuations a block can collect
constexpr uint32_t kFar = 0xFFFFFFFFu;                   // a distance of 32 bits or more

// The largest of the warp's values, and the sum of its values below 2^48, by 32-bit reductions.
__device__ __forceinline__ long long warp_max(long long v) {
  const int32_t hi = __reduce_max_sync(0xffffffffu, (int32_t)(v >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (int32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return (long long)((unsigned long long)(uint32_t)hi << 32 | lo);
}
__device__ __forceinline__ unsigned long long warp_sum48(unsigned long long v) {
  const uint32_t lo = __reduce_add_sync(0xffffffffu, (uint32_t)v & 0xFFFFFFu);
  const uint32_t hi = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 24));
  return ((unsigned long long)hi << 24) + lo;
}

__device__ __forceinline__ unsigned long long distance(long long m, long long l) {
  const unsigned long long d = (unsigned long long)m - (unsigned long long)l;
  return d < kMaxDistance ? d : kMaxDistance;
}

// Polls for the phase with the given parity; whether it came.
__device__ __forceinline__ bool came(uint64_t* bar, uint32_t parity, uint32_t polls) {
  for (uint32_t i = 0; i < polls; ++i)
    if (mb_try(bar, parity)) return true;
  return false;
}

// The rows' nearest continuations, a cluster a row (and then the next but as many as there are
// clusters), whose blocks split the vocabulary.  A block reads its logits once into registers
// (once a pass where they are more): the maximum, pushed to the other blocks; the distances, cut
// to 32 bits, and the sum of their exponentials, from a table in shared memory (gathered through
// L1 the kernel takes 63 us for 512 rows of 32,000, against 41 to 46); then a bound that at least
// `beams` threads' least distances meet, by their bit length and the three bits below it, so that
// what meets it (a few more than `beams`, unless there are many ties) contains the block's
// nearest, which are ranked by counting.  More than kFound at the bound, or a bound past 32
// bits: one after the other, by index.  A block whose wait for the maxima runs out gives the row up:
// it marks its sum as lost, so that the merge fails the row's search, and waits once more for what
// is on its way to it, so that it neither leaves before nor takes it for the next row's.  Where rows are many the instructions bound it (512 rows of
// 32,000: 131 MB in 46 us, 2.9 TB/s, half of the issue slots), where they are few the chain of
// these steps.
template <bool ONE>
__global__ void __launch_bounds__(kBeamThreads, kBeamBlocks) k_beam_row(const BeamParams p) {
  __shared__ uint32_t table[4097], found_d[kFound], found_i[kFound], bits[33], below[8], red_i[kBeamWarps], n_found;
  __shared__ unsigned long long red[kBeamWarps], peaks[2][8 * kBeamWarps];
  __shared__ uint64_t arrived[2];  // the cluster's maxima of a row, in turn
  __shared__ int gave_up;          // a warp's wait for this row's maxima ran out
  const uint32_t S = p.split, rank = blockIdx.x % S, clusters = gridDim.x / S;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = p.beams, rows = p.groups * k;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the merge waits for this grid's end)
  const uint32_t per = (p.vocab + S - 1) / S, v0 = min(p.vocab, rank * per), n = min(p.vocab, v0 + per) - v0;
  const uint32_t want = min(k, n);  // (at most 64: each thread has one)
  constexpr uint32_t kWord = 8;
  if (tid < 33) bits[tid] = 0;
  if (tid == 0) {
    gave_up = 0;
    for (int i = 0; i < 2; ++i) {
      mb_init(arrived + i, 1);
      mb_expect_tx(arrived + i, S * kBeamWarps * kWord);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // every block of the cluster runs, its barriers ready, before another writes into its memory
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  for (uint32_t i = tid; i < 4097; i += kBeamThreads) table[i] = min(__ldg(p.exp_tab + i), 1u << 30);
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  uint32_t pushed = 0;  // rows whose maxima went around
  for (uint32_t row = blockIdx.x / S; row < rows; row += clusters) {
    const long long* l = reinterpret_cast<const long long*>(p.logits) + row * p.stride + v0;
    long long x[kPer];
    auto load = [&](uint32_t base) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const uint32_t i = base + j * kBeamThreads + tid;
        x[j] = i < n ? __ldg(l + i) : LLONG_MIN;
      }
    };
    if (ONE) load(0);
    const long long old = p.scores[row];
    const bool ended = p.done[row] != 0, alive = old > kDeadScore && old < -kDeadScore;
    unsigned long long* ld = p.list_d + ((size_t)row * S + rank) * k;
    uint32_t* lt = p.list_token + ((size_t)row * S + rank) * k;
    if (!alive || ended) {  // (for every block of the cluster)
      for (uint32_t i = tid; i < k; i += kBeamThreads) {
        ld[i] = alive && rank == 0 && i == 0 ? 0 : ~0ull;
        lt[i] = p.vocab;
      }
      if (tid == 0) p.part_z[(size_t)row * S + rank] = 0;
      continue;
    }
    long long m = LLONG_MIN;
    for (uint32_t base = 0; base < (ONE ? 1 : n); base += kRound) {
      if (!ONE) load(base);
#pragma unroll
      for (int j = 0; j < kPer; ++j) m = max(m, x[j]);
    }
    m = warp_max(m);
    __syncthreads();  // the row before is done with shared memory
    if (tid < 8) below[tid] = 0;  // (the block's next barriers come before their use)
    if (tid == 0) n_found = 0;
    const uint32_t turn = pushed & 1u;
    if (lane < S) {  // each warp's maximum to block `lane`, completing on that block's barrier
      uint32_t a = (uint32_t)__cvta_generic_to_shared(&peaks[turn][rank * kBeamWarps + warp]);
      uint32_t bar = (uint32_t)__cvta_generic_to_shared(arrived + turn);
      asm("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(a) : "r"(lane));
      asm("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(bar) : "r"(lane));
      asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(a), "l"(m), "r"(bar)
                   : "memory");
    }
    // A block sends its next row's maxima once it has read this one's, and waits for all: so
    // those of the row after next find this turn's words read.
    if (!came(arrived + turn, (pushed >> 1) & 1u, p.polls)) {
      gave_up = 1;
      came(arrived + turn, (pushed >> 1) & 1u, kTcPoll);
    }
    ++pushed;
    if (tid == 0) mb_expect_tx(arrived + turn, S * kBeamWarps * kWord);
#pragma unroll
    for (uint32_t i = 0; i < 8 * kBeamWarps; i += 32)
      if (i + lane < S * kBeamWarps) m = max(m, (long long)peaks[turn][i + lane]);
    m = warp_max(m);

    // (a place without a logit is far: it adds the table's last entry to the sum, taken off again)
    uint32_t d[kPer], least = kFar;
    auto distances = [&](uint32_t base) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const unsigned long long w = (unsigned long long)m - (unsigned long long)x[j];
        d[j] = w >> 32 || base + j * kBeamThreads + tid >= n ? kFar : (uint32_t)w;
      }
    };
    if (ONE) distances(0);
    unsigned long long z = 0;
    for (uint32_t base = 0; base < (ONE ? 1 : n); base += kRound) {
      if (!ONE) {
        load(base);
        distances(base);
      }
#pragma unroll
      for (int j = 0; j < kPer; j += 2) {  // (entries are at most 2^30: two add up in 32 bits)
        z += table[min(d[j] >> 8, 4096u)] + table[min(d[j + 1] >> 8, 4096u)];
        least = min(least, min(d[j], d[j + 1]));
      }
      const uint32_t rest = n - min(n, base + tid), held = min((rest + kBeamThreads - 1) / kBeamThreads, (uint32_t)kPer);
      z -= (unsigned long long)(kPer - held) * table[4096];
    }
    // the bound: the bit length at which enough least distances are counted, then three bits more
    const bool mine = tid < n;
    const uint32_t length = 32 - __clz((int)least), three = length >= 4 ? least >> (length - 4) & 7u : 0;
    if (mine) atomicAdd(bits + length, 1u);
    __syncthreads();
    const bool lost = gave_up != 0;
    // each warp scans the counts: bit lengths 0 .. 31 (at = 32: none of them)
    const uint32_t count = bits[lane];
    uint32_t upto = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t w = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += w;
    }
    const uint32_t enough = __ballot_sync(0xffffffffu, upto >= want);
    const uint32_t at = enough ? __ffs((int)enough) - 1 : 32;
    const uint32_t before = __shfl_sync(0xffffffffu, upto - count, at & 31u);  // (for at < 32)
    if (mine && length == at) atomicAdd(below + three, 1u);
    z = warp_sum48(z);
    if (lane == 0) red[warp] = z;
    __syncthreads();
    // The counts have been read, and this row's last barrier and the next one's first come before
    // they are added to again: the wait for the maxima in between orders the pushed words alone.
    if (tid < 33) bits[tid] = 0;
    if (tid == 0) gave_up = 0;
    uint32_t bound = at >= 32 ? kFar : (1u << at) - 1;
    if (at >= 4 && at < 32) {
      uint32_t sum = lane < 8 ? below[lane] : 0;
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) {
        const uint32_t w = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += w;
      }
      const uint32_t met = __ballot_sync(0xffffffffu, lane < 8 && before + sum >= want);  // (lane 7 does)
      bound = (uint32_t)((8 + __ffs((int)met)) << (at - 4)) - 1;
    }
    if (tid == 0) {
      z = 0;
      for (int w = 0; w < kBeamWarps; ++w) z += red[w];
      p.part_z[(size_t)row * S + rank] = lost ? kLost : z;
    }
    for (uint32_t base = 0; base < (ONE ? 1 : n) && least <= bound; base += kRound) {
      if (!ONE) {
        load(base);
        distances(base);
      }
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (d[j] <= bound && d[j] != kFar) {  // (at the bound kFar the list is not used)
          const uint32_t to = atomicAdd(&n_found, 1u);
          if (to < kFound) {
            found_d[to] = d[j];
            found_i[to] = v0 + base + j * kBeamThreads + tid;
          }
        }
      }
    }
    __syncthreads();
    const uint32_t nf = n_found;
    const uint32_t some = lost ? 0 : want;
    for (uint32_t i = some + tid; i < k; i += kBeamThreads) {
      ld[i] = ~0ull;
      lt[i] = p.vocab;
    }
    if (some == 0) continue;
    if (nf <= kFound && bound != kFar) {
      for (uint32_t i = tid; i < nf; i += kBeamThreads) {
        const uint32_t e = found_d[i], token = found_i[i];
        uint32_t rank_of = 0;
#pragma unroll 4
        for (uint32_t j = 0; j < nf; ++j) rank_of += found_d[j] < e || (found_d[j] == e && found_i[j] < token);
        if (rank_of < k) {
          ld[rank_of] = e;
          lt[rank_of] = token;
        }
      }
      continue;
    }
    unsigned long long last_d = 0;
    uint32_t last_i = 0;
    for (uint32_t c = 0; c < want; ++c) {
      unsigned long long bd = ~0ull;
      uint32_t bi = p.vocab;
      for (uint32_t i = tid; i < n; i += kBeamThreads) {
        const unsigned long long w = distance(m, __ldg(l + i));
        if ((c == 0 || w > last_d || (w == last_d && v0 + i > last_i)) && w < bd) {
          bd = w;
          bi = v0 + i;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long od = __shfl_xor_sync(0xffffffffu, bd, o);
        const uint32_t oi = __shfl_xor_sync(0xffffffffu, bi, o);
        if (od < bd || (od == bd && oi < bi)) {
          bd = od;
          bi = oi;
        }
      }
      __syncthreads();  // (the round before has been read)
      if (lane == 0) {
        red[warp] = bd;
        red_i[warp] = bi;
      }
      __syncthreads();
      for (int w = 0; w < kBeamWarps; ++w)
        if (red[w] < bd || (red[w] == bd && red_i[w] < bi)) {
          bd = red[w];
          bi = red_i[w];
        }
      last_d = bd;
      last_i = bi;
      if (tid == 0) {
        ld[c] = bd;
        lt[c] = bi;
      }
    }
  }
}

// The best of a search's lists together, a block a search.  The `beams`-th best head of the lists
// bounds what can be chosen: the entries that meet it (those of equal scores among them) are
// ranked by counting.  More than kChosen of them: one warp walks the lists, taking the best
// head each time.  Lists come in the order of beam and token, so the lower list wins a tie.
// The latency of its steps bounds it: 10.6 us for 64 searches of 8 beams.
constexpr int kMergeThreads = 256;
constexpr uint32_t kChosen = 512;
__global__ void __launch_bounds__(kMergeThreads) k_beam_merge(const BeamParams p) {
  __shared__ long long base[64], head[64 * 8], chosen[kChosen];
  __shared__ uint32_t entry[kChosen], token[kChosen], n_chosen;
  __shared__ uint16_t at[64 * 8];
  __shared__ long long least;
  const uint32_t g = blockIdx.x, tid = threadIdx.x, k = p.beams, S = p.split, first = g * k, lists = k * S;
  if (tid == 0) {
    n_chosen = 0;
    least = LLONG_MIN;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const unsigned long long* ld = p.list_d + (size_t)first * lists;
  const uint32_t* lt = p.list_token + (size_t)first * lists;
  int lost = 0;
  for (uint32_t b = tid; b < k; b += kMergeThreads) {
    unsigned long long z = 0;
#pragma unroll
    for (uint32_t r = 0; r < 8; ++r) {
      const unsigned long long part = r < S ? __ldcg(p.part_z + (size_t)(first + b) * S + r) : 0;
      lost |= part == kLost;
      z += part;
    }
    base[b] = p.scores[first + b] - log_sum(z);  // (an ended beam's z is zero, and so its logarithm)
  }
  // outcome n: entry e (list * beams + place) with token t
  auto put = [&](uint32_t n, long long score, uint32_t e, uint32_t t) {
    p.scores_out[first + n] = score;
    p.parent[first + n] = first + e / (k * S);
    p.token[first + n] = t < p.vocab ? t : p.done_token;
    p.done_out[first + n] = t == p.vocab || ((p.flags & CK_FLAG_STOP_TOKENS) && (t == 1 || t == 2));
  };
  auto put_none = [&](uint32_t n, uint8_t done) {
    p.scores_out[first + n] = LLONG_MIN;
    p.parent[first + n] = CK_NO_PAGE;
    p.token[first + n] = p.done_token;
    p.done_out[first + n] = done;
  };
  // heads, and the first entries (all of them, where beams are few), asked for at once
  const uint32_t all = lists * k;
  unsigned long long mine[2], early_d[2];
  uint32_t early_t[2];
#pragma unroll
  for (uint32_t u = 0; u < 2; ++u) {
    const uint32_t i = tid + u * kMergeThreads;
    mine[u] = i < lists ? __ldcg(ld + (size_t)i * k) : ~0ull;
    early_d[u] = i < all ? __ldcg(ld + i) : ~0ull;
    early_t[u] = i < all ? __ldcg(lt + i) : 0;
  }
  if (__syncthreads_or(lost)) {  // what is left of the search is not its selection
    for (uint32_t n = tid; n < k; n += kMergeThreads) put_none(n, CK_BEAM_FAILED);
    return;
  }
#pragma unroll
  for (uint32_t u = 0; u < 2; ++u) {
    const uint32_t i = tid + u * kMergeThreads;
    if (i >= lists) continue;
    head[i] = mine[u] == ~0ull ? LLONG_MIN : base[i / S] - (long long)mine[u];
    at[i] = 0;
  }
  __syncthreads();
  for (uint32_t i = tid; i < lists; i += kMergeThreads) {
    const long long h = head[i];
    uint32_t rank_of = 0;
#pragma unroll 4
    for (uint32_t j = 0; j < lists; ++j) rank_of += head[j] > h || (head[j] == h && j < i);
    if (rank_of == k - 1) least = h;  // (one list has this rank)
  }
  __syncthreads();
  const long long bound = least;
  auto choose = [&](uint32_t e, unsigned long long d, uint32_t t) {
    const long long v = d == ~0ull ? LLONG_MIN : base[e / (k * S)] - (long long)d;
    if (v == LLONG_MIN || v < bound) return;
    const uint32_t to = atomicAdd(&n_chosen, 1u);
    if (to < kChosen) {
      chosen[to] = v;
      entry[to] = e;
      token[to] = t;
    }
  };
#pragma unroll
  for (uint32_t u = 0; u < 2; ++u)
    if (tid + u * kMergeThreads < all) choose(tid + u * kMergeThreads, early_d[u], early_t[u]);
  for (uint32_t e = tid + 2 * kMergeThreads; e < all; e += kMergeThreads)
    if (head[e / k] >= bound) choose(e, __ldcg(ld + e), __ldcg(lt + e));
  __syncthreads();
  const uint32_t nc = n_chosen;
  if (nc <= kChosen) {
    for (uint32_t i = tid; i < nc; i += kMergeThreads) {
      const long long v = chosen[i];
      const uint32_t e = entry[i];
      uint32_t rank_of = 0;
#pragma unroll 4
      for (uint32_t j = 0; j < nc; ++j) rank_of += chosen[j] > v || (chosen[j] == v && entry[j] < e);
      if (rank_of < k) put(rank_of, v, e, token[i]);
    }
    for (uint32_t n = nc + tid; n < k; n += kMergeThreads) put_none(n, 0);
    return;
  }
  if (tid >= 32) return;
  for (uint32_t n = 0; n < k; ++n) {
    long long best = LLONG_MIN;
    uint32_t from = ~0u;
    for (uint32_t i = tid; i < lists; i += 32)
      if (head[i] > best) {
        best = head[i];
        from = i;
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const long long ov = __shfl_xor_sync(0xffffffffu, best, o);
      const uint32_t of = __shfl_xor_sync(0xffffffffu, from, o);
      if (ov > best || (ov == best && of < from)) {
        best = ov;
        from = of;
      }
    }
    const bool some = from != ~0u;
    if (tid == (some ? from & 31 : 0)) {
      if (some) {
        const uint32_t e = from * k + at[from];
        put(n, best, e, __ldcg(lt + e));
        const uint32_t c = ++at[from];
        const unsigned long long d = c < k ? __ldcg(ld + (size_t)from * k + c) : ~0ull;
        head[from] = d == ~0ull ? LLONG_MIN : base[from / S] - (long long)d;
      } else {
        put_none(n, 0);
      }
    }
    __syncwarp();
  }
}

// Blocks of a cluster: until each holds its logits in registers, eight at most.
uint32_t beam_split(uint32_t vocab) {
  uint32_t S = 1;
  while (S < 8 && S * kRound < vocab) S *= 2;
  return S;
}

// Clusters of S blocks that are resident at once, looked up once for each S.
template <bool ONE>
cudaError_t resident_clusters(cudaLaunchConfig_t* cfg, uint32_t S, const DeviceFacts& f, uint32_t* out) {
  static std::atomic<int> known[64][9];
  int n = known[f.dev][S].load(std::memory_order_relaxed);
  if (n == 0) {
    cfg->gridDim = dim3(S);
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, k_beam_row<ONE>, cfg);
    if (e != cudaSuccess) return e;
    known[f.dev][S].store(n, std::memory_order_relaxed);
  }
  *out = (uint32_t)std::max(n, 1);
  return cudaSuccess;
}

cudaError_t launch_beam(const BeamParams& p, cudaStream_t s) {
  DeviceFacts f;
  cudaError_t e = device_facts(&f);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kBeamThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool one = (p.vocab + p.split - 1) / p.split <= kRound;
  uint32_t clusters;
  e = one ? resident_clusters<true>(&cfg, p.split, f, &clusters) : resident_clusters<false>(&cfg, p.split, f, &clusters);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(std::min(p.groups * p.beams, clusters) * p.split);
  e = one ? cudaLaunchKernelEx(&cfg, k_beam_row<true>, p) : cudaLaunchKernelEx(&cfg, k_beam_row<false>, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(p.groups);
  cfg.blockDim = dim3(kMergeThreads);
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  return cudaLaunchKernelEx(&cfg, k_beam_merge, p);
}

bool beam_sizes_ok(uint32_t groups, uint32_t beams, uint32_t vocab) {
  return groups >= 1 && beams >= 1 && beams <= 64 && vocab >= 1 && vocab <= (1u << 20) &&
         (uint64_t)groups * beams <= 65536;
}
// Scratch: partial sums, distances, tokens.
struct BeamLayout {
  uint64_t z, d, token, size;
};
BeamLayout beam_layout(uint64_t rows, uint32_t beams, uint32_t vocab) {
  const uint64_t lists = rows * beam_split(vocab);
  BeamLayout w;
  w.z = 0;
  w.d = align256(8 * lists);
  w.token = w.d + align256(8 * lists * beams);
  w.size = w.token + align256(4 * lists * beams);
  return w;
}

}  // namespace
}  // namespace ck

using namespace ck;

extern "C" {

int64_t ck_host_log_sum(uint64_t z) { return log_sum(z); }

int ck_set_beam_wait_limit(uint32_t polls) {
  g_wait_limit.store(polls, std::memory_order_relaxed);
  return CK_OK;
}

int ck_beam_work(uint32_t groups, uint32_t beams, uint32_t vocab, size_t* out) {
  if (!out || !beam_sizes_ok(groups, beams, vocab)) return CK_INVALID_ARGUMENT;
  *out = beam_layout((uint64_t)groups * beams, beams, vocab).size;
  return CK_OK;
}

int ck_beam_select(const int64_t* dev_logits, size_t logits_stride, uint32_t groups, uint32_t beams,
                   uint32_t vocab, const int64_t* dev_scores, const uint8_t* dev_done,
                   const uint32_t* dev_exp, uint32_t flags, uint32_t done_token, int64_t* dev_scores_out,
                   uint32_t* dev_parent, uint32_t* dev_token, uint8_t* dev_done_out, void* dev_work,
                   size_t work_len, void* stream) {
  size_t need;
  if (const int rc = ck_beam_work(groups, beams, vocab, &need)) return rc;
  if (!dev_logits || !dev_scores || !dev_done || !dev_exp || !dev_scores_out || !dev_parent || !dev_token ||
      !dev_done_out || !dev_work)
    return CK_INVALID_ARGUMENT;
  if (logits_stride < vocab || logits_stride >> 40 || done_token >= vocab || (flags & ~CK_FLAG_STOP_TOKENS))
    return CK_INVALID_ARGUMENT;
  const uint64_t rows = (uint64_t)groups * beams;
  const void* in[] = {dev_logits, dev_scores, dev_done, dev_exp};
  const uint64_t in_bytes[] = {8 * ((rows - 1) * logits_stride + vocab), 8 * rows, rows, 4 * 4097};
  const void* out[] = {dev_scores_out, dev_parent, dev_token, dev_done_out, dev_work};
  const uint64_t out_bytes[] = {8 * rows, 4 * rows, 4 * rows, rows, work_len};
  const uintptr_t out_align[] = {8, 4, 4, 1, 256};
  if (!aligned_to(dev_logits, 8) || !aligned_to(dev_scores, 8) || !aligned_to(dev_exp, 4)) return CK_INVALID_ARGUMENT;
  for (int o = 0; o < 5; ++o) {
    if (!aligned_to(out[o], out_align[o])) return CK_INVALID_ARGUMENT;
    for (int i = 0; i < 4; ++i)
      if (overlaps(out[o], out_bytes[o], in[i], in_bytes[i])) return CK_INVALID_ARGUMENT;
    for (int i = 0; i < o; ++i)
      if (overlaps(out[o], out_bytes[o], out[i], out_bytes[i])) return CK_INVALID_ARGUMENT;
  }
  if (work_len < need) return CK_BUFFER_TOO_SMALL;
  BeamParams p = {};
  p.logits = dev_logits;
  p.stride = logits_stride;
  p.groups = groups;
  p.beams = beams;
  p.vocab = vocab;
  p.flags = flags;
  p.done_token = done_token;
  p.scores = dev_scores;
  p.done = dev_done;
  p.exp_tab = dev_exp;
  p.scores_out = dev_scores_out;
  p.parent = dev_parent;
  p.token = dev_token;
  p.done_out = dev_done_out;
  const BeamLayout w = beam_layout(rows, beams, vocab);
  uint8_t* work = static_cast<uint8_t*>(dev_work);
  p.split = beam_split(vocab);
  const uint32_t limit = g_wait_limit.load(std::memory_order_relaxed);
  p.polls = limit ? limit - 1 : kTcPoll;
  p.part_z = reinterpret_cast<unsigned long long*>(work + w.z);
  p.list_d = reinterpret_cast<unsigned long long*>(work + w.d);
  p.list_token = reinterpret_cast<uint32_t*>(work + w.token);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  CKP_CUDA(launch_beam(p, s));
  return CK_OK;
}

}  // extern "C"
