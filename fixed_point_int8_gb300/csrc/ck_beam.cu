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
  long long* cand_score;   // [rows][beams], descending; a dead entry is the lowest int64
  uint32_t* cand_token;    // [rows][beams]; `vocab`: an ended beam
};

constexpr int kBeamThreads = 512, kBeamWarps = kBeamThreads / 32;

__device__ __forceinline__ unsigned long long distance(long long m, long long l) {
  const unsigned long long d = (unsigned long long)m - (unsigned long long)l;
  return d < kMaxDistance ? d : kMaxDistance;
}

// A row's `beams` nearest continuations, one block a row: the maximum, the sum of exponentials,
// then one continuation after the other, each the nearest behind the one before.
__global__ void __launch_bounds__(kBeamThreads) k_beam_row(const BeamParams p) {
  __shared__ unsigned long long red[kBeamWarps];
  __shared__ uint32_t red_i[kBeamWarps];
  const uint32_t row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long old = p.scores[row];
  const bool alive = old > kDeadScore && old < -kDeadScore;
  long long* cs = p.cand_score + (size_t)row * p.beams;
  uint32_t* ct = p.cand_token + (size_t)row * p.beams;
  if (!alive || p.done[row]) {
    for (uint32_t i = tid; i < p.beams; i += kBeamThreads) {
      cs[i] = alive && i == 0 ? old : LLONG_MIN;
      ct[i] = p.vocab;
    }
    return;
  }
  const long long* l = reinterpret_cast<const long long*>(p.logits) + row * p.stride;
  long long m = LLONG_MIN;
  for (uint32_t i = tid; i < p.vocab; i += kBeamThreads) m = max(m, l[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red[warp] = (unsigned long long)m;
  __syncthreads();
  for (int w = 0; w < kBeamWarps; ++w) m = max(m, (long long)red[w]);
  __syncthreads();
  unsigned long long z = 0;
  for (uint32_t i = tid; i < p.vocab; i += kBeamThreads) {
    const unsigned long long d = distance(m, l[i]) >> 8;
    z += __ldg(p.exp_tab + (d < 4096 ? d : 4096));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  if (lane == 0) red[warp] = z;
  __syncthreads();
  z = 0;
  for (int w = 0; w < kBeamWarps; ++w) z += red[w];
  __syncthreads();
  const long long base = old - log_sum(z);
  unsigned long long last_d = 0;
  uint32_t last_i = 0;
  for (uint32_t n = 0; n < p.beams; ++n) {
    unsigned long long bd = ~0ull;
    uint32_t bi = p.vocab;
    for (uint32_t i = tid; i < p.vocab; i += kBeamThreads) {
      const unsigned long long d = distance(m, l[i]);
      if ((n == 0 || d > last_d || (d == last_d && i > last_i)) && d < bd) {
        bd = d;
        bi = i;
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
    __syncthreads();
    last_d = bd;
    last_i = bi;
    if (tid == 0) {
      cs[n] = bi < p.vocab ? base - (long long)bd : LLONG_MIN;
      ct[n] = bi;
    }
  }
}

// The best of a search's beams together, a warp a search: lane j walks the lists of rows j and
// j + 32, and the warp takes the best head each time.
__global__ void __launch_bounds__(32) k_beam_merge(const BeamParams p) {
  const uint32_t g = blockIdx.x, lane = threadIdx.x, first = g * p.beams;
  uint32_t at[2] = {0, 0};
  for (uint32_t n = 0; n < p.beams; ++n) {
    long long best = LLONG_MIN;
    uint32_t row = ~0u;
#pragma unroll
    for (uint32_t u = 0; u < 2; ++u) {
      const uint32_t b = lane + 32 * u;
      if (b >= p.beams || at[u] >= p.beams) continue;
      const long long v = p.cand_score[(size_t)(first + b) * p.beams + at[u]];
      if (v > best) {
        best = v;
        row = b;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const long long ov = __shfl_xor_sync(0xffffffffu, best, o);
      const uint32_t orow = __shfl_xor_sync(0xffffffffu, row, o);
      if (ov > best || (ov == best && orow < row)) {
        best = ov;
        row = orow;
      }
    }
    const bool some = row != ~0u;
    if (lane == (some ? row & 31 : 0)) {
      uint32_t token = p.done_token;
      bool done = false;
      if (some) {
        const uint32_t t = p.cand_token[(size_t)(first + row) * p.beams + (row < 32 ? at[0] : at[1])];
        row < 32 ? ++at[0] : ++at[1];
        done = t == p.vocab || ((p.flags & CK_FLAG_STOP_TOKENS) && (t == 1 || t == 2));
        if (t < p.vocab) token = t;
      }
      p.scores_out[first + n] = best;
      p.parent[first + n] = some ? first + row : CK_NO_PAGE;
      p.token[first + n] = token;
      p.done_out[first + n] = done;
    }
    __syncwarp();
  }
}

bool beam_sizes_ok(uint32_t groups, uint32_t beams, uint32_t vocab) {
  return groups >= 1 && beams >= 1 && beams <= 64 && vocab >= 1 && vocab <= (1u << 20) &&
         (uint64_t)groups * beams <= 65536;
}
uint64_t beam_scores_bytes(uint64_t rows, uint32_t beams) { return align256(8 * rows * beams); }

}  // namespace
}  // namespace ck

using namespace ck;

extern "C" {

int64_t ck_host_log_sum(uint64_t z) { return log_sum(z); }

int ck_beam_work(uint32_t groups, uint32_t beams, uint32_t vocab, size_t* out) {
  if (!out || !beam_sizes_ok(groups, beams, vocab)) return CK_INVALID_ARGUMENT;
  const uint64_t rows = (uint64_t)groups * beams;
  *out = beam_scores_bytes(rows, beams) + align256(4 * rows * beams);
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
  p.cand_score = static_cast<long long*>(dev_work);
  p.cand_token = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(dev_work) + beam_scores_bytes(rows, beams));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  k_beam_row<<<(uint32_t)rows, kBeamThreads, 0, s>>>(p);
  k_beam_merge<<<groups, 32, 0, s>>>(p);
  CKP_CUDA(cudaGetLastError());
  return CK_OK;
}

}  // extern "C"
