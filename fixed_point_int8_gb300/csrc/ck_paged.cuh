// Shared by the operators of the paged cache and of beam search: argument checks, the device's
// properties, and how a kernel finds a row's sequence and a position's page.
#pragma once
#include <atomic>

#include "ck_internal.cuh"

namespace ck {

#define CKP_CUDA(call)                                   \
  do {                                                   \
    if ((call) != cudaSuccess) return CK_CUDA_ERROR;     \
  } while (0)

constexpr uint32_t kMaxPositions = (1u << 20) - 1;  // 20 bits of an error key

inline bool aligned_to(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
inline bool pow2_in(uint32_t v, uint32_t lo, uint32_t hi) { return v >= lo && v <= hi && (v & (v - 1)) == 0; }
inline uint32_t log2_of(uint32_t v) {
  uint32_t s = 0;
  while ((1u << s) < v) ++s;
  return s;
}
inline bool overlaps(const void* a, uint64_t na, const void* b, uint64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na != 0 && nb != 0 && x < y + nb && y < x + na;
}

inline bool cache_ok(const ck_paged_cache* c) {
  return c && pow2_in(c->head_dim, 4, 128) && pow2_in(c->page, 8, 256) && c->layers >= 1 && c->layers <= 4095 &&
         c->kv_heads >= 1 && c->kv_heads <= 4096 && c->pages >= 1 && c->pages <= (1u << 24);
}
inline bool pools_ok(const ck_paged_cache* c) {
  return cache_ok(c) && c->dev_k && c->dev_v && aligned_to(c->dev_k, 16) && aligned_to(c->dev_v, 16);
}
inline bool batch_sizes_ok(const ck_paged_batch* b) {
  return b && b->seqs >= 1 && b->seqs <= 65535 && b->rows >= 1 && b->rows <= (1u << 20) && b->stride >= 1 &&
         b->stride <= (1u << 17) && b->max_new >= 1 && b->max_new <= b->rows && b->max_len >= 1 &&
         b->max_len <= kMaxPositions;
}
inline bool batch_ok(const ck_paged_batch* b) {
  return batch_sizes_ok(b) && b->dev_start && b->dev_len && b->dev_table && b->dev_status &&
         aligned_to(b->dev_start, 4) && aligned_to(b->dev_len, 4) && aligned_to(b->dev_table, 4) &&
         aligned_to(b->dev_status, 8);
}

// Whether a call's output (or scratch) of n bytes lies on the pools, or on them or the batch's arrays.
inline bool on_pools(const void* p, uint64_t n, const ck_paged_cache& c) {
  const uint64_t page = 4ull * c.layers * c.kv_heads * c.page * c.head_dim;  // at most 2^41 bytes
  const uint64_t pool = std::min<uint64_t>(c.pages, (1ull << 62) / page) * page;
  return overlaps(p, n, c.dev_k, pool) || overlaps(p, n, c.dev_v, pool);
}
inline bool on_batch(const void* p, uint64_t n, const ck_paged_cache& c, const ck_paged_batch& b) {
  return on_pools(p, n, c) || overlaps(p, n, b.dev_start, 4ull * (b.seqs + 1)) ||
         overlaps(p, n, b.dev_len, 4ull * b.seqs) || overlaps(p, n, b.dev_table, 4ull * b.seqs * b.stride) ||
         overlaps(p, n, b.dev_status, 8ull * b.seqs);
}

// Streaming multiprocessors and opt-in shared memory of the current device, looked up once.
struct DeviceFacts {
  int dev, sms, optin;
};
inline cudaError_t device_facts(DeviceFacts* f) {
  static std::atomic<int> sms[64], optin[64];
  cudaError_t e = cudaGetDevice(&f->dev);
  if (e != cudaSuccess) return e;
  if (f->dev < 0 || f->dev >= 64) return cudaErrorInvalidDevice;
  f->sms = sms[f->dev].load(std::memory_order_relaxed);
  f->optin = optin[f->dev].load(std::memory_order_relaxed);
  if (f->sms == 0 || f->optin == 0) {
    if ((e = cudaDeviceGetAttribute(&f->sms, cudaDevAttrMultiProcessorCount, f->dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&f->optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, f->dev)) != cudaSuccess)
      return e;
    sms[f->dev].store(f->sms, std::memory_order_relaxed);
    optin[f->dev].store(f->optin, std::memory_order_relaxed);
  }
  return cudaSuccess;
}

// A pass of a paged batch through a model's layers (ck_batch.cu): its scratch, and its kernels.
size_t paged_pass_bytes(const PrefillModel& m, uint32_t cap, size_t attn_bytes);
cudaError_t enqueue_paged_pass(const PrefillModel& m, const ck_paged_cache* cache, const ck_paged_batch* batch,
                               const uint32_t* tokens, int64_t* logits, size_t logits_stride, size_t attn_bytes,
                               uint8_t* work, cudaStream_t s);

// The pool and the batch as kernels take them.
struct PoolView {
  int32_t* k;
  int32_t* v;
  uint32_t pages, layers, kv_heads, page_shift, hd, layer;
};
inline PoolView pool_view(const ck_paged_cache& c, uint32_t layer) {
  return {c.dev_k, c.dev_v, c.pages, c.layers, c.kv_heads, log2_of(c.page), c.head_dim, layer};
}
struct BatchView {
  const uint32_t* start;
  const uint32_t* len;
  const uint32_t* table;
  unsigned long long* status;
  uint32_t seqs, rows, stride, max_new, max_len;
};
inline BatchView batch_view(const ck_paged_batch& b) {
  return {b.dev_start, b.dev_len, b.dev_table, reinterpret_cast<unsigned long long*>(b.dev_status),
          b.seqs, b.rows, b.stride, b.max_new, b.max_len};
}

// First word of (page id, layer, kv head): that head's positions of the page follow one another.
__device__ __forceinline__ size_t page_word(const PoolView& p, uint32_t id, uint32_t kvh) {
  return (((((size_t)id * p.layers + p.layer) * p.kv_heads + kvh) << p.page_shift)) * p.hd;
}

// The sequence whose rows hold `row`, for every thread of a block, or `seqs` when none does: the
// ascending starts at or below the row are counted, a block's width at a time.
__device__ __forceinline__ uint32_t block_find_seq(const BatchView& b, uint32_t row) {
  uint32_t s = 0;
  for (uint32_t base = 0; base < b.seqs; base += blockDim.x) {
    const uint32_t i = base + threadIdx.x;
    s += (uint32_t)__syncthreads_count(i < b.seqs && b.start[i + 1] <= row);
  }
  return s;
}

struct Sequence {
  uint32_t s, first, count, len;
  bool ok;  // within the bounds the launch was sized by
  // Whether the row, at or behind the first, is one of the sequence's: where the starts do not ascend
  // it may not be, and its position would lie behind the sequence's pages.
  __device__ __forceinline__ bool holds(uint32_t row) const { return row - first < count; }
};
__device__ __forceinline__ Sequence load_sequence(const BatchView& b, uint32_t s, uint32_t page_shift) {
  Sequence q;
  q.s = s;
  q.first = b.start[s];
  const uint32_t end = b.start[s + 1];
  q.count = end >= q.first ? end - q.first : 0;
  q.len = b.len[s];
  q.ok = end >= q.first && end <= b.rows && q.count <= b.max_new && q.len <= b.max_len &&
         q.len <= ((uint64_t)b.stride << page_shift);
  return q;
}
__device__ __forceinline__ void note(const BatchView& b, uint32_t s, uint64_t key) {
  atomicMin(b.status + s, (unsigned long long)key);
}

}  // namespace ck
