// Beam search's selection over beams and vocabulary ("Sampling", with the sum pass at
// temperature one): every beam's continuations by their distance to its largest logit, the
// logarithm of its sum of exponentials, and the best of all beams together.
#include "ck_paged.cuh"

namespace ck {
namespace {

constexpr long long kDeadScore = -(1ll << 61);
constexpr unsigned long long kMaxDistance = 1ull << 62;

// ln(z / 2^30), 16 fraction bits (0 below 2^30): z = 2^n y with y in [1, 2), ln y = 2 atanh t
// of t = (y - 1) / (y + 1) <= 1/3, its series to t^15 (the next term is below 2^-28).
__host__ __device__ inline int64_t log_sum(uint64_t z) {
  if (z < (1ull << 30)) z = 1ull << 30;
  uint32_t n = 0;
  while (n < 33 && (z >> n) >> 31) ++n;
  const uint64_t y = z >> n, one = 1ull << 30;
  const uint64_t t = ((y - one) << 30) / (y + one), T = (t * t) >> 30;
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
  unsigned long long* part_z;     // [rows][split]
  unsigned long long* list_d;     // [rows][split][beams]
  uint32_t* list_token;           // [rows][split][beams]
};

constexpr int kBeamThreads = 256, kBeamWarps = kBeamThreads / 32;
constexpr int kPer = 16;                                 // logits a thread holds
constexpr uint32_t kRound = kPer * kBeamThreads;         // logits a block takes at once
constexpr uint32_t kFound = 512;                         // continuations a block can collect

__device__ __forceinline__ unsigned long long distance(long long m, long long l) {
  const unsigned long long d = (unsigned long long)m - (unsigned long long)l;
  return d < kMaxDistance ? d : kMaxDistance;
}

// A row's nearest continuations, by a cluster of blocks that split the vocabulary.  A block
// reads its logits once into registers (once a pass where they are more): the maximum, pushed to
// the other blocks; the sum of exponentials and each thread's least distance; then a bound that
// at least `beams` threads' least distances meet, found by counting from the highest bit down,
// so that what meets it (a few more than `beams`, unless there are many ties) contains the
// block's nearest, which are ranked by counting.  More than kFound at the bound: one after the
// other, by index.
template <bool ONE>
__global__ void __launch_bounds__(kBeamThreads, 4) k_beam_row(const BeamParams p) {
  __shared__ unsigned long long red[kBeamWarps], found_d[kFound], peaks[8];
  __shared__ uint32_t red_i[kBeamWarps], found_i[kFound], n_found;
  const uint32_t S = p.split, rank = blockIdx.x % S, row = blockIdx.x / S;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = p.beams;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the merge waits for this grid's end)
  const uint32_t per = (p.vocab + S - 1) / S, v0 = min(p.vocab, rank * per), n = min(p.vocab, v0 + per) - v0;
  const long long* l = reinterpret_cast<const long long*>(p.logits) + row * p.stride + v0;
  long long x[kPer];
  auto load = [&](uint32_t base) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const uint32_t i = base + j * kBeamThreads + tid;
      x[j] = i < n ? __ldg(l + i) : LLONG_MIN;
    }
  };
  const long long old = p.scores[row];
  const bool ended = p.done[row] != 0, alive = old > kDeadScore && old < -kDeadScore;
  unsigned long long* ld = p.list_d + (size_t)blockIdx.x * k;
  uint32_t* lt = p.list_token + (size_t)blockIdx.x * k;
  if (!alive || ended) {  // (the whole cluster leaves)
    for (uint32_t i = tid; i < k; i += kBeamThreads) {
      ld[i] = alive && rank == 0 && i == 0 ? 0 : ~0ull;
      lt[i] = p.vocab;
    }
    if (tid == 0) p.part_z[blockIdx.x] = 0;
    return;
  }
  if (ONE) load(0);
  long long m = LLONG_MIN;
  for (uint32_t base = 0; base < (ONE ? 1 : n); base += kRound) {
    if (!ONE) load(base);
#pragma unroll
    for (int j = 0; j < kPer; ++j) m = max(m, x[j]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red[warp] = (unsigned long long)m;
  if (tid == 0) n_found = 0;
  __syncthreads();
  if (tid < S) {
    for (int w = 0; w < kBeamWarps; ++w) m = max(m, (long long)red[w]);
    uint32_t a = (uint32_t)__cvta_generic_to_shared(peaks + rank);
    asm("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(a) : "r"(tid));
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(m) : "memory");
  }
  // (after this nothing reads or writes another block's memory)
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  for (uint32_t r = 0; r < S; ++r) m = max(m, (long long)peaks[r]);

  unsigned long long z = 0, least = ~0ull;
  for (uint32_t base = 0; base < (ONE ? 1 : n); base += kRound) {
    if (!ONE) load(base);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (base + j * kBeamThreads + tid >= n) continue;
      const unsigned long long d = distance(m, x[j]), i = d >> 8;
      z += __ldg(p.exp_tab + (i < 4096 ? i : 4096));
      least = d < least ? d : least;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  if (lane == 0) red[warp] = z;
  const uint32_t want = min(k, n);  // (at most 64: each thread has one)
  unsigned long long bound = ~0ull;
  if (want != 0) {
    uint32_t lo = 0, hi = 63;  // bit lengths: 63 holds every distance
    while (lo < hi) {
      const uint32_t mid = (lo + hi) / 2;
      if ((uint32_t)__syncthreads_count(least < (1ull << mid)) >= want)
        hi = mid;
      else
        lo = mid + 1;
    }
    bound = (1ull << lo) - 1;
#pragma unroll 1
    for (uint32_t s = 2; s <= 4 && lo >= s; ++s) {
      const unsigned long long cut = bound - (1ull << (lo - s));
      if ((uint32_t)__syncthreads_count(least <= cut) >= want) bound = cut;
    }
  }
  __syncthreads();
  if (tid == 0) {
    z = 0;
    for (int w = 0; w < kBeamWarps; ++w) z += red[w];
    p.part_z[blockIdx.x] = z;
  }
  for (uint32_t base = 0; base < (ONE ? 1 : n); base += kRound) {
    if (!ONE) load(base);
    if (least > bound) continue;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const uint32_t i = base + j * kBeamThreads + tid;
      const unsigned long long d = distance(m, x[j]);
      if (i < n && d <= bound) {
        const uint32_t at = atomicAdd(&n_found, 1u);
        if (at < kFound) {
          found_d[at] = d;
          found_i[at] = v0 + i;
        }
      }
    }
  }
  __syncthreads();
  const uint32_t nf = n_found;
  for (uint32_t i = want + tid; i < k; i += kBeamThreads) {
    ld[i] = ~0ull;
    lt[i] = p.vocab;
  }
  if (nf <= kFound) {
    for (uint32_t i = tid; i < nf; i += kBeamThreads) {
      const unsigned long long d = found_d[i];
      const uint32_t at = found_i[i];
      uint32_t before = 0;
#pragma unroll 4
      for (uint32_t j = 0; j < nf; ++j) before += found_d[j] < d || (found_d[j] == d && found_i[j] < at);
      if (before < k) {
        ld[before] = d;
        lt[before] = at;
      }
    }
    return;
  }
  unsigned long long last_d = 0;
  uint32_t last_i = 0;
  for (uint32_t c = 0; c < want; ++c) {
    unsigned long long bd = ~0ull;
    uint32_t bi = p.vocab;
    for (uint32_t base = 0; base < (ONE ? 1 : n); base += kRound) {
      if (!ONE) load(base);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const uint32_t i = base + j * kBeamThreads + tid;
        const unsigned long long d = distance(m, x[j]);
        if (i < n && (c == 0 || d > last_d || (d == last_d && v0 + i > last_i)) && d < bd) {
          bd = d;
          bi = v0 + i;
        }
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

// The best of a search's lists together, a block a search: the rows' bases (score less lnZ) and,
// where they fit, the lists into shared memory; then one warp walks them, each lane the lists
// lane, lane + 32, ... (in the order of beam and token), taking the best head each time.
constexpr int kMergeThreads = 128;
constexpr uint32_t kMergeLists = 2048;  // entries of the lists kept in shared memory
__global__ void __launch_bounds__(kMergeThreads) k_beam_merge(const BeamParams p) {
  __shared__ long long base[64];
  __shared__ uint16_t at[64 * 8];
  __shared__ unsigned long long sd[kMergeLists];
  __shared__ uint32_t st[kMergeLists];
  const uint32_t g = blockIdx.x, lane = threadIdx.x & 31, k = p.beams, S = p.split, first = g * k;
  const uint32_t lists = k * S, all = lists * k;
  for (uint32_t i = threadIdx.x; i < lists; i += kMergeThreads) at[i] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const unsigned long long* ld = p.list_d + (size_t)first * S * k;
  const uint32_t* lt = p.list_token + (size_t)first * S * k;
  const bool here = all <= kMergeLists;
  for (uint32_t i = threadIdx.x; here && i < all; i += kMergeThreads) {
    sd[i] = __ldcg(ld + i);
    st[i] = __ldcg(lt + i);
  }
  for (uint32_t b = threadIdx.x; b < k; b += kMergeThreads) {
    unsigned long long z = 0;
#pragma unroll
    for (uint32_t r = 0; r < 8; ++r) z += r < S ? __ldcg(p.part_z + (size_t)(first + b) * S + r) : 0;
    base[b] = p.scores[first + b] - log_sum(z);  // (an ended beam's z is zero, and so its logarithm)
  }
  __syncthreads();
  if (threadIdx.x >= 32) return;
  for (uint32_t n = 0; n < k; ++n) {
    long long best = LLONG_MIN;
    uint32_t from = ~0u;
    for (uint32_t i = lane; i < lists; i += 32) {
      const uint32_t c = at[i];
      if (c >= k) continue;
      const unsigned long long d = here ? sd[i * k + c] : __ldcg(ld + i * k + c);
      if (d == ~0ull) continue;
      const long long v = base[i / S] - (long long)d;
      if (v > best) {
        best = v;
        from = i;
      }
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
    if (lane == (some ? from & 31 : 0)) {
      uint32_t token = p.done_token;
      bool done = false;
      if (some) {
        const uint32_t e = from * k + at[from], t = here ? st[e] : __ldcg(lt + e);
        ++at[from];
        done = t == p.vocab || ((p.flags & CK_FLAG_STOP_TOKENS) && (t == 1 || t == 2));
        if (t < p.vocab) token = t;
      }
      p.scores_out[first + n] = best;
      p.parent[first + n] = some ? first + from / S : CK_NO_PAGE;
      p.token[first + n] = token;
      p.done_out[first + n] = done;
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

cudaError_t launch_beam(const BeamParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.groups * p.beams * p.split);
  cfg.blockDim = dim3(kBeamThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = (p.vocab + p.split - 1) / p.split <= kRound ? cudaLaunchKernelEx(&cfg, k_beam_row<true>, p)
                                                                    : cudaLaunchKernelEx(&cfg, k_beam_row<false>, p);
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
  const void* in[] = {dev_logits, dev_scores, dev_done};
  const uint64_t in_bytes[] = {8 * ((rows - 1) * logits_stride + vocab), 8 * rows, rows};
  const void* out[] = {dev_scores_out, dev_parent, dev_token, dev_done_out, dev_work};
  const uint64_t out_bytes[] = {8 * rows, 4 * rows, 4 * rows, rows, work_len};
  const uintptr_t out_align[] = {8, 4, 4, 1, 256};
  if (!aligned_to(dev_logits, 8) || !aligned_to(dev_scores, 8) || !aligned_to(dev_exp, 4)) return CK_INVALID_ARGUMENT;
  for (int o = 0; o < 5; ++o) {
    if (!aligned_to(out[o], out_align[o])) return CK_INVALID_ARGUMENT;
    for (int i = 0; i < 3; ++i)
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
  p.part_z = reinterpret_cast<unsigned long long*>(work + w.z);
  p.list_d = reinterpret_cast<unsigned long long*>(work + w.d);
  p.list_token = reinterpret_cast<uint32_t*>(work + w.token);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  CKP_CUDA(launch_beam(p, s));
  return CK_OK;
}

}  // extern "C"
